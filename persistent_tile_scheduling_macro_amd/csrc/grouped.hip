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

// tile_rows(bm): upper bound of the tile rows of height bm over all experts.
template <class F>
int launch(pgemm_ctx* h, grouped::Args a, bool direct, int64_t mean_rows, F tile_rows, int dtype, bool grad, bool nk) {
  const int body = direct && mean_rows >= 192 ? grouped::kPingPong : grouped::kAnyAlignment;
  const int tile = body == grouped::kPingPong ? 256 : 128;
  a.n_n = (a.N + tile - 1) / tile;
  int64_t grid = tile_rows(tile) * a.n_n;
  if (grid > INT32_MAX - 8) return fail(h, PGEMM_ERR_UNSUPPORTED, "more than 2^31 output tiles");
  if (body == grouped::kPingPong) grid = grid < h->cus ? grid : h->cus; // persistent, one workgroup a CU
  else if (!grad) grid = (grid + 7) / 8 * 8;
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  const grouped::kernel_fn kern = dtype == PGEMM_F16 ? grouped::pick_f16(body, grad, nk) : grouped::pick_bf16(body, grad, nk);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(body == grouped::kPingPong ? 512 : 256), 0, h->stream, a);
  return launch_status(h, "grouped product");
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
  return launch(h, a, direct, R / E, [&](int bm) { return R / bm + E + 1; }, dtype, false, layout == PGEMM_B_NK);
}

int pgemm_grouped_weight_grad(pgemm_handle_t h, const void* a_rows, int64_t lda, const void* b_rows, int64_t ldb,
                              const int32_t* offsets, void* c, int64_t R, int64_t E, int64_t I, int64_t J, int dtype) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  const int rc = check(h, R, E, I, J, lda, ldb, dtype);
  if (rc != PGEMM_OK) return rc;
  if (I == 0 || J == 0) return PGEMM_OK;
  if (!offsets || !c || (R > 0 && (!a_rows || !b_rows))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
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
  const bool direct = I % 8 == 0 && J % 8 == 0 && lda % 8 == 0 && ldb % 8 == 0 && lda <= kMaxDirectStride &&
                      ldb <= kMaxDirectStride && aligned16(a_rows) && aligned16(b_rows) && aligned16(c);
  return launch(h, a, direct, R / E, [&](int bm) { return E * ((I + bm - 1) / bm); }, dtype, true, false);
}

} // extern "C"
