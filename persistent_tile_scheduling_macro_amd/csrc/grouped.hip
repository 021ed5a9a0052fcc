// Entry points of the products of rows sorted by expert.
#include "context.h"
#include "grouped.h"

using namespace pgemm;

namespace {

constexpr int64_t kMaxSize = (int64_t)1 << 30;

int check(pgemm_ctx* h, int64_t R, int64_t E, int64_t K, int64_t N, int64_t lda, int64_t ldb, int dtype) {
  if (R < 0 || K < 0 || N < 0 || E < 1 || lda < 0 || ldb < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "sizes R=%lld E=%lld, %lld x %lld, row strides %lld, %lld", (long long)R,
                (long long)E, (long long)K, (long long)N, (long long)lda, (long long)ldb);
  if (dtype != PGEMM_F16 && dtype != PGEMM_BF16)
    return fail(h, PGEMM_ERR_INVALID_ARG, "dtype %d is not fp16 or bf16", dtype);
  if (R > kMaxSize || K > kMaxSize || N > kMaxSize) return fail(h, PGEMM_ERR_UNSUPPORTED, "sizes must not exceed 2^30");
  if (E > moe::kMaxExperts)
    return fail(h, PGEMM_ERR_UNSUPPORTED, "E=%lld experts, at most %d", (long long)E, moe::kMaxExperts);
  return PGEMM_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }

static_assert(grouped::kAnyAlignment == PGEMM_GROUPED_ANY && grouped::kPingPong == PGEMM_GROUPED_PINGPONG &&
                  grouped::kFew16 == PGEMM_GROUPED_FEW16 && grouped::kFew16Wide == PGEMM_GROUPED_FEW16_WIDE &&
                  grouped::kFew32Wide == PGEMM_GROUPED_FEW32_WIDE && grouped::kFewGrad == PGEMM_GROUPED_FEW_GRAD,
              "the query's numbers are the bodies'");

// Tile of a body: rows, columns, threads.
struct Shape { int bm, bn, threads; };
Shape shape_of(int body, bool nk) {
  switch (body) {
    case grouped::kPingPong: return {256, 256, 512};
    case grouped::kFew16: return {16, nk ? 16 : 64, 512};
    case grouped::kFew16Wide: return {16, nk ? 32 : 64, 512};
    case grouped::kFew32Wide: return {32, nk ? 32 : 64, 512};
    case grouped::kFewGrad: return {128, 128, 512};
    default: return {128, 128, 256};
  }
}

// The body of the rows form. How many rows each expert has only the device
// knows; with their mean, a body's time is estimated as rounds of workgroups
// (so many of them run at once) times what one takes, or the time its reads
// of the matrices take, if that is more:
//   body     at once  a workgroup takes, us                     reads at
//   few      512      4 + 0.0018 K (32 rows x 32 columns)       4.8 TB/s
//   any      512      4 + 0.020 K; from 256 down 4 + 0.016 K    4 TB/s
//   ping     256      4 + 0.0184 K                              4 TB/s
// fitted to measured calls of K = 256 .. 4096, N = 64 .. 4096, 1 .. 64 experts
// and 64 .. 16000 rows. Examples (few, any, ping-pong; us): one expert, 4096 x
// 512, 256 rows 12, 61, 79, 4000 rows 62, 69, 80; eight experts, 1024 x 2048,
// 1600 rows 46, 22, 27, 8000 rows 188, 62, 55; eight experts, 4096 x 4096,
// 8000 rows 888, 400, 277.
int pick_rows_body(const grouped::Args& a, bool direct, bool nk) {
  const double experts = a.R < a.E ? a.R : a.E, mean = a.R / experts, K = a.K;
  struct Cost { double groups, reads; };
  auto cost = [&](int body) {
    const Shape t = shape_of(body, nk);
    double row_tiles = a.E == 1 ? __builtin_ceil(mean / t.bm) : mean / t.bm + 0.5; // an expert's last one is half full on average
    if (row_tiles < 1) row_tiles = 1;
    const bool few = t.bm < 128; // reads a matrix again for every row tile, the others find it in the L2
    return Cost{experts * row_tiles * ((a.N + t.bn - 1) / t.bn), experts * (few ? row_tiles / 4.8e6 : 1 / 4.0e6) * K * a.N * 2};
  };
  auto longer = [](double x, double y) { return x > y ? x : y; };
  int best = grouped::kAnyAlignment;
  Cost c = cost(best);
  const double crowd = c.groups < 256 ? 0 : c.groups > 512 ? 1 : c.groups / 256 - 1; // two on a CU
  double least = longer(__builtin_ceil(c.groups / 512) * (4 + (0.016 + 0.004 * crowd) * K), c.reads);
  if (direct) {
    c = cost(grouped::kPingPong);
    const double t = longer(__builtin_ceil(c.groups / 256) * (4 + 0.0184 * K), c.reads);
    if (t < least) best = grouped::kPingPong, least = t;
  }
  if (K > 0 && (nk || a.N >= 4)) {
    // 16 rows where they hold an expert's; two column blocks share the reads of x where that leaves enough workgroups
    int body = grouped::kFew32Wide;
    if (mean <= 8) body = cost(grouped::kFew16Wide).groups >= 512 ? grouped::kFew16Wide : grouped::kFew16;
    c = cost(body);
    if (longer(__builtin_ceil(c.groups / 512) * (4 + 0.0018 * K), c.reads) < least) best = body;
  }
  return best;
}

// Body and pieces of the gradient form, by the same kind of estimate: rounds of workgroups times what one
// takes (4 us and 1.28 us for 64 rows of a 128 x 128 tile with two on a CU, 1.18 us of a 256 x 256 tile),
// and what the pieces' sums cost on their way through memory. A piece has 192 rows at least. (One expert,
// 32768 rows: 64 x 64 647 us in one piece, 512 x 512 653 us, 2048 x 2048 718 us.)
struct GradPlan { int body; int64_t pieces; };
GradPlan plan_grad(int64_t R, int64_t E, int64_t I, int64_t J) {
  // The body for few rows, where its many small steps were faster (us, against the better of the others): 32
  // experts, 2048 x 1536, of 31 rows 39, 64 rows 47 (58), 94 rows 63 (64), 128 rows 77 (75); eight of 200 rows, 1024 x
  // 1024 12 (16), 1023 x 1023 17 (15); one of 400 rows, 512 x 512 9 (18).
  // Odd sizes, whose edges it moves inside the loop, only with few rows or very few tiles: ten of 480 rows, 144 x 1184
  // 22 (25), 145 x 1183 34 (24).
  const int64_t tiles_128 = E * ((I + 127) / 128) * ((J + 127) / 128), rows = R / E;
  const bool even = I % 8 == 0 && J % 8 == 0;
  if (rows <= 96 || (even && rows <= 256 && tiles_128 <= 768) || (rows <= 512 && tiles_128 <= (even ? 256 : 32)))
    return {grouped::kFewGrad, 1};
  GradPlan best = {grouped::kAnyAlignment, 1};
  double least = 1e30;
  const double mean = (double)R / E;
  for (int body : {grouped::kAnyAlignment, grouped::kPingPong}) {
    if (body == grouped::kPingPong && (I % 8 || J % 8)) continue;
    const int64_t bm = body == grouped::kPingPong ? 256 : 128, at_once = body == grouped::kPingPong ? 256 : 512;
    const int64_t tiles = E * ((I + bm - 1) / bm) * ((J + bm - 1) / bm);
    if (tiles == 0) return best;
    int64_t fill = at_once / tiles, most = R / E / 192;
    if (fill > most) fill = most;
    if (fill > 64) fill = 64;
    for (int64_t s : {(int64_t)1, fill}) {
      if (s < 1) continue;
      const double rounds = (double)((tiles * s + at_once - 1) / at_once);
      const double t = rounds * (4 + mean / s / 64 * (body == grouped::kPingPong ? 1.18 : 1.28)) +
                       (s > 1 ? 3 + 8e-6 / 4.5 * s * E * I * J : 0);
      if (t < least) {
        least = t;
        best = {body, s};
      }
    }
  }
  return best;
}

// Plan of the gradient form for operands that can, or cannot, be copied directly.
GradPlan plan_grad_for(int64_t R, int64_t E, int64_t I, int64_t J, bool direct) {
  GradPlan p = plan_grad(R, E, I, J);
  if (!direct && p.body != grouped::kFewGrad) p.body = grouped::kAnyAlignment; // the workspace is the same either way
  return p;
}

// tile_rows(bm): upper bound of the tile rows of height bm over all experts.
template <class F>
int launch(pgemm_ctx* h, grouped::Args a, int body, F tile_rows, int dtype, bool grad, bool nk) {
  const Shape t = shape_of(body, nk);
  a.n_n = (a.N + t.bn - 1) / t.bn;
  int64_t grid = tile_rows(t.bm) * a.n_n;
  if (grid > INT32_MAX - 8) return fail(h, PGEMM_ERR_UNSUPPORTED, "more than 2^31 output tiles");
  a.most_tiles = (int)grid;
  if (body == grouped::kPingPong) grid = grid < h->cus ? grid : h->cus; // persistent, one workgroup a CU
  else if (!grad) grid = (grid + 7) / 8 * 8;
  if (grid * t.threads > UINT32_MAX) // threads of a launch
    return fail(h, PGEMM_ERR_UNSUPPORTED, "%lld output tiles are more than one launch takes", (long long)grid);
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  const bool f16 = dtype == PGEMM_F16;
  hipError_t e = enqueue(h->stream, dim3((unsigned)grid), dim3(t.threads),
                         f16 ? grouped::pick_f16(body, grad, nk) : grouped::pick_bf16(body, grad, nk), a);
  if (e == hipSuccess && a.split > 1) {
    const bool shared = a.split >= 8;
    const int64_t sums = (int64_t)a.E * a.M * ((a.N + 7) / 8), per = shared ? 32 : 256;
    e = enqueue(h->stream, dim3((unsigned)((sums + per - 1) / per)), dim3(256),
                f16 ? grouped::join_f16(shared) : grouped::join_bf16(shared), a);
  }
  return launch_status(h, e, "grouped product");
}

// Row strides up to which a tile's 32-bit offsets reach its last row (256 rows of 2-byte elements below 2^31).
constexpr int64_t kMaxDirectStride = (int64_t)1 << 21;

} // namespace

extern "C" {

int pgemm_grouped_run(pgemm_handle_t h, const void* x, int64_t ldx, const void* w, const int32_t* offsets, void* y,
                      int64_t R, int64_t E, int64_t K, int64_t N, int layout, int dtype) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  const int rc = check(h, R, E, K, N, ldx, 0, dtype);
  if (rc != PGEMM_OK) return rc;
  if (layout != PGEMM_B_KN && layout != PGEMM_B_NK) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown layout %d", layout);
  if (R == 0 || N == 0) return PGEMM_OK;
  if (!offsets || !y || (K > 0 && (!x || !w))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  grouped::Args a = {};
  a.a = static_cast<const uint16_t*>(x);
  a.b = static_cast<const uint16_t*>(w);
  a.lda = ldx;
  a.ldb = layout == PGEMM_B_NK ? K : N;
  a.b_expert = K * N;
  a.offsets = offsets;
  a.c = static_cast<uint16_t*>(y);
  a.R = (int)R;
  a.E = (int)E;
  a.K = (int)K;
  a.N = (int)N;
  const bool direct = K % 8 == 0 && N % 8 == 0 && ldx % 8 == 0 && ldx <= kMaxDirectStride && a.ldb <= kMaxDirectStride &&
                      aligned16(x) && aligned16(w) && aligned16(y);
  // every expert, and the rows of none, may leave one tile partly filled
  const bool nk = layout == PGEMM_B_NK;
  return launch(h, a, pick_rows_body(a, direct, nk), [&](int bm) { return R / bm + E + 1; }, dtype, false, nk);
}

int pgemm_grouped_query(int64_t R, int64_t E, int64_t K, int64_t N, int layout, int wide, int* body) {
  if (!body || R < 1 || E < 1 || K < 1 || N < 1 || (layout != PGEMM_B_KN && layout != PGEMM_B_NK)) return PGEMM_ERR_INVALID_ARG;
  if (R > kMaxSize || K > kMaxSize || N > kMaxSize || E > moe::kMaxExperts) return PGEMM_ERR_UNSUPPORTED;
  grouped::Args a = {};
  a.R = (int)R;
  a.E = (int)E;
  a.K = (int)K;
  a.N = (int)N;
  *body = pick_rows_body(a, wide && K % 8 == 0 && N % 8 == 0, layout == PGEMM_B_NK);
  return PGEMM_OK;
}

int pgemm_grouped_weight_grad_query(int64_t R, int64_t E, int64_t I, int64_t J, int wide, int* body, int* pieces) {
  if (!body || !pieces || R < 1 || E < 1 || I < 1 || J < 1) return PGEMM_ERR_INVALID_ARG;
  if (R > kMaxSize || I > kMaxSize || J > kMaxSize || E > moe::kMaxExperts) return PGEMM_ERR_UNSUPPORTED;
  const GradPlan p = plan_grad_for(R, E, I, J, wide && I % 8 == 0 && J % 8 == 0);
  *body = p.body;
  *pieces = (int)p.pieces;
  return PGEMM_OK;
}

int pgemm_grouped_weight_grad_workspace(int64_t R, int64_t E, int64_t I, int64_t J, int64_t* bytes) {
  if (!bytes || R < 0 || E < 1 || I < 0 || J < 0) return PGEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (R > kMaxSize || I > kMaxSize || J > kMaxSize || E > moe::kMaxExperts) return PGEMM_ERR_UNSUPPORTED;
  const int64_t s = plan_grad(R, E, I, J).pieces;
  if (s > 1) *bytes = s * E * I * ((J + 7) / 8 * 8) * (int64_t)sizeof(float);
  return PGEMM_OK;
}

int pgemm_grouped_weight_grad(pgemm_handle_t h, const void* a_rows, int64_t lda, const void* b_rows, int64_t ldb,
                              const int32_t* offsets, void* c, int64_t R, int64_t E, int64_t I, int64_t J, int dtype,
                              void* work, int64_t work_bytes) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  int rc = check(h, R, E, I, J, lda, ldb, dtype);
  if (rc != PGEMM_OK) return rc;
  if (I == 0 || J == 0) return PGEMM_OK;
  if (!offsets || !c || (R > 0 && (!a_rows || !b_rows))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  int64_t need = 0;
  rc = pgemm_grouped_weight_grad_workspace(R, E, I, J, &need);
  if (rc != PGEMM_OK) return rc;
  if (work_bytes < need || (need && !aligned16(work)) || (need && !work))
    return fail(h, PGEMM_ERR_INVALID_ARG, "workspace of %lld bytes at %p, %lld at a multiple of 16 are needed",
                (long long)work_bytes, work, (long long)need);
  grouped::Args a = {};
  a.a = static_cast<const uint16_t*>(a_rows);
  a.b = static_cast<const uint16_t*>(b_rows);
  a.lda = lda;
  a.ldb = ldb;
  a.offsets = offsets;
  a.c = static_cast<uint16_t*>(c);
  a.R = (int)R;
  a.E = (int)E;
  a.M = (int)I;
  a.N = (int)J;
  a.part = static_cast<float*>(work);
  const bool direct = I % 8 == 0 && J % 8 == 0 && lda % 8 == 0 && ldb % 8 == 0 && lda <= kMaxDirectStride &&
                      ldb <= kMaxDirectStride && aligned16(a_rows) && aligned16(b_rows) && aligned16(c);
  const GradPlan plan = plan_grad_for(R, E, I, J, direct);
  a.split = (int)plan.pieces;
  return launch(h, a, plan.body, [&](int bm) { return E * a.split * ((I + bm - 1) / bm); }, dtype, true, false);
}

} // extern "C"
