// Entry points of the linear layer.
#include "context.h"
#include "dense.h"

using namespace pgemm;

namespace {

using dense::Args;

constexpr int64_t kMaxSize = (int64_t)1 << 30;
// Row strides up to which a tile's 32-bit offsets reach its last row (256 rows of 2-byte elements below 2^31).
constexpr int64_t kMaxDirectStride = (int64_t)1 << 21;

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

// Scratch handed out piece by piece; with a null base it only counts.
struct Scratch {
  char* base;
  int64_t used = 0;
  template <class T>
  T* take(int64_t count) {
    const int64_t at = used;
    used += (count * (int64_t)sizeof(T) + 255) / 256 * 256;
    return base ? reinterpret_cast<T*>(base + at) : nullptr;
  }
};

static_assert((int)dense::kFew8 == (int)PGEMM_DENSE_FEW8 && (int)dense::kFew16 == (int)PGEMM_DENSE_FEW16 && (int)dense::kFew32 == (int)PGEMM_DENSE_FEW32 &&
                  (int)dense::kTile64 == (int)PGEMM_DENSE_TILE64 && (int)dense::kTile128 == (int)PGEMM_DENSE_TILE128 &&
                  (int)dense::kTile128Pair == (int)PGEMM_DENSE_TILE128_PAIR && (int)dense::kPing == (int)PGEMM_DENSE_PINGPONG,
              "the query's numbers are the bodies'");
static_assert((int)act::kNone == (int)PGEMM_ACT_NONE && (int)act::kRelu == (int)PGEMM_ACT_RELU && (int)act::kGelu == (int)PGEMM_ACT_GELU &&
                  (int)act::kGeluTanh == (int)PGEMM_ACT_GELU_TANH && (int)act::kSilu == (int)PGEMM_ACT_SILU,
              "the header's numbers are the activations'");

struct Plan { int body; int split; double time; };

struct Tile { int bm, bn; };
Tile tile_of(int body) { return body == dense::kPing ? Tile{256, 256} : body == dense::kTile64 ? Tile{64, 128} : Tile{128, 128}; }

// The bodies' times in us on 256 CUs, fitted to 2878 measured calls at 240 sizes of 1 .. 8192 rows and 64 .. 8192 columns and
// sums (replayed from a graph, bf16, operands changing from call to call; all of them in profiles/dense_layer_rules.txt); the
// rule below was 2% slower than the fastest in the geometric mean, 36% at worst. Examples (the times of few, tile 64, tile 128, pair, ping-pong, each with its
// best number of pieces): 24 x 4096 x 4096 9, 14, 16, 18, 27; 512 x 4096 x 8192 -, 71, 43, 53, 59; 4099 x 2056 x 1024
// -, -, 36, 31, 36; 8192 x 8192 x 4096 -, -, 615, 545, 455.
//
// few: base + the longer of rounds of 256 workgroups, each `start` and `step` for each k, and reading W for every
// group of rows at `rate` TB/s.
struct FewCost { double base, start, step, rate; };
constexpr FewCost kFewCost[2][2][3] = { // K x N, N x K; plain, gated; 8, 16, 32 rows
    {{{2.4, 0.4, 0.00315, 6.5}, {3.0, 0.0, 0.00315, 4.0}, {3.3, 0.0, 0.0037, 3.4}},
     {{3.2, 0.0, 0.0049, 2.8}, {4.9, 0.5, 0.0038, 6.3}, {5.1, 0.0, 0.0045, 3.8}}},
    {{{1.6, 0.6, 0.00096, 5.4}, {2.1, 0.65, 0.0010, 6.0}, {2.5, 0.45, 0.0010, 5.5}},
     {{3.4, 0.0, 0.0009, 6.5}, {1.5, 1.1, 0.00175, 6.0}, {1.9, 1.0, 0.0022, 5.3}}}};
// tiles: base + rounds of workgroups, each `start` and for each 64 k `step`, or `full` when every CU has one (two); at
// least the operands' bytes at 5 TB/s; pieces cost `join` and `join_sum` for each million partial sums.
struct TileCost { double base, start, step, full, join, join_sum; };
constexpr TileCost kTileCost[4] = {{2.5, 1.9, 0.285, 0.51, 1.9, 1.87},  // kTile64
                                   {2.8, 3.2, 0.38, 0.525, 1.2, 1.86},  // kTile128
                                   {5.1, 0.0, 0.695, 1.04, 0.7, 2.15},  // kTile128Pair
                                   {9.9, 0.45, 1.19, 1.63, 0.0, 1.25}}; // kPing

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int few_rows(int body) { return body == dense::kFew8 ? 8 : body == dense::kFew16 ? 16 : 32; }
int few_columns(bool nk) { return nk ? 16 : 64; } // of y

double few_time(int body, int64_t M, int64_t N, int64_t K, bool nk, bool gated) {
  const FewCost& c = kFewCost[nk][gated][body - dense::kFew8];
  const double groups = (double)ceil_div(M, few_rows(body));
  const double work = (double)ceil_div((int64_t)groups * ceil_div(N, few_columns(nk)), 256) * (c.start + c.step * K);
  const double reads = groups * K * (gated ? 2 : 1) * N * 2e-6 / c.rate;
  return c.base + (work > reads ? work : reads);
}
double tile_time(int body, int64_t rows, int64_t columns, int64_t sum, int64_t pieces) {
  const TileCost& c = kTileCost[body - dense::kTile64];
  const Tile t = tile_of(body);
  const int64_t groups = ceil_div(rows, t.bm) * ceil_div(columns, t.bn) * pieces;
  const int64_t slots = body == dense::kTile128Pair ? 512 : 256;
  double load = groups / 256.0 - (slots == 512);
  load = load < 0 ? 0 : load > 1 ? 1 : load;
  const double work = (double)ceil_div(groups, slots) * (c.start + (double)ceil_div(sum, 64) / pieces * (c.step + (c.full - c.step) * load));
  const double reads = 2.0 * ((double)rows * sum + (double)sum * columns + (double)rows * columns) / 5e6;
  const double join = pieces > 1 ? c.join + 0.15 * pieces + c.join_sum * 1e-6 * pieces * rows * columns : 0;
  return c.base + (work > reads ? work : reads) + join;
}

// Tries a tile body with the numbers of pieces that leave each at least two steps of 64.
void try_tiles(int body, int64_t rows, int64_t columns, int64_t sum, double extra, Plan* best) {
  const int64_t steps = ceil_div(sum, 64);
  for (int pieces : {1, 2, 3, 4, 6, 8, 12}) {
    if (pieces > 1 && (pieces * 2 > steps || (body == dense::kTile128Pair && pieces > 4))) break;
    const Tile t = tile_of(body);
    if (pieces > 1 && ceil_div(rows, t.bm) * ceil_div(columns, t.bn) * pieces > 1024) break;
    const double time = extra + tile_time(body, rows, columns, sum, pieces);
    if (time < best->time) *best = {body, pieces, time};
  }
}

// Body and pieces of a product of M x K with K x N (gated: 2N) columns. pad_x, pad_w: sizes whose rows the tile bodies
// need moved first (a launch of 3 us and a pass over the operand).
Plan plan_rows(int64_t M, int64_t N, int64_t K, bool nk, bool gated, bool pad_x, bool pad_w) {
  const int64_t C = gated ? 2 * N : N;
  Plan best = {dense::kTile128, 1, 1e30};
  const double extra = pad_x * (3 + 1e-6 * M * K) + pad_w * (3 + 1e-6 * C * K);
  if (N % 8 == 0) try_tiles(dense::kPing, M, C, K, extra, &best);
  try_tiles(dense::kTile128, M, C, K, extra, &best);
  try_tiles(dense::kTile128Pair, M, C, K, extra, &best);
  if (M <= 512) try_tiles(dense::kTile64, M, C, K, extra, &best);
  if (M <= 128 && (nk || N >= 4)) {
    for (int body : {(int)dense::kFew8, (int)dense::kFew16, (int)dense::kFew32}) {
      if (M > 16 ? body == dense::kFew8 : few_rows(body) / 2 >= M && body > dense::kFew8) continue;
      const double time = few_time(body, M, N, K, nk, gated);
      if (time < best.time) best = {body, 1, time};
    }
  }
  return best;
}

// The same for c [I][J] = a^T b over R rows.
Plan plan_grad(int64_t R, int64_t I, int64_t J) {
  Plan best = {dense::kTile128, 1, 1e30};
  if (J % 8 == 0) try_tiles(dense::kPing, I, J, R, 0, &best);
  try_tiles(dense::kTile128, I, J, R, 0, &best);
  try_tiles(dense::kTile128Pair, I, J, R, 0, &best);
  return best;
}

// Both products of a backward pass, dx [M][K] over C and dw over M, as tiles of 128 x 128 in one launch, if that is faster
// than one after the other (the second launch waits some 3 us for the first to drain). The workgroups are laid on the
// card's slots as the hardware does, the longer ones first. Over 40 sizes of 128 .. 8192 rows, 88 .. 3725 columns the
// gradients took with the rule 2% longer than with the best body and pieces in the geometric mean, 18% at worst, in two
// launches 31% (profiles/dense_layer_rules.txt).
struct Both { int body, split_x, split_w; bool dw_first; };
bool plan_both(int64_t M, int64_t K, int64_t C, bool nk, const Plan& dx, const Plan& dw, Both* best) {
  if (dx.body <= dense::kFew32) return false;
  const int64_t I = nk ? C : K, J = nk ? K : C;
  const int64_t steps_x = ceil_div(C, 64), steps_w = ceil_div(M, 64);
  const int64_t tiles_x = ceil_div(M, 128) * ceil_div(K, 128), tiles_w = ceil_div(I, 128) * ceil_div(J, 128);
  if (tiles_x + tiles_w > 1024) return false; // each fills the card by itself
  double least = dx.time + dw.time + 3;
  bool found = false;
  for (int body : {(int)dense::kTile128, (int)dense::kTile128Pair}) {
    const TileCost& c = kTileCost[body - dense::kTile64];
    const int64_t slots = body == dense::kTile128Pair ? 512 : 256;
    for (int px : {1, 2, 3, 4, 6, 8, 12}) {
      if (px > 1 && (px * 2 > steps_x || tiles_x * px > 1024 || (slots == 512 && px > 4))) break;
      for (int pw : {1, 2, 3, 4, 6, 8, 12}) {
        if (pw > 1 && (pw * 2 > steps_w || tiles_w * pw > 1024 || (slots == 512 && pw > 4))) break;
        const int64_t groups_x = tiles_x * px, groups_w = tiles_w * pw;
        if ((px > 1 || pw > 1) && groups_x + groups_w > 2 * slots) break; // pieces are for few tiles
        double load = (groups_x + groups_w) / 256.0 - (slots == 512);
        load = load < 0 ? 0 : load > 1 ? 1 : load;
        const double step = c.step + (c.full - c.step) * load;
        const double time_x = c.start + (double)steps_x / px * step, time_w = c.start + (double)steps_w / pw * step;
        const bool dw_first = time_w > time_x;
        const int64_t first = dw_first ? groups_w : groups_x, then = dw_first ? groups_x : groups_w;
        const double longer = dw_first ? time_w : time_x, shorter = dw_first ? time_x : time_w;
        // after the first: `late` slots are busy a round longer than the others
        const int64_t late = first % slots;
        double early_end = (double)(first / slots) * longer, late_end = late ? early_end + longer : early_end;
        double end = late_end;
        for (int64_t left = then; left > 0;) {
          const bool take_late = late && late_end < early_end;
          double& at = take_late ? late_end : early_end;
          at += shorter;
          end = at > end ? at : end;
          left -= take_late ? late : slots - late;
        }
        const double elements_x = (double)M * K, elements_w = (double)I * J;
        const double reads = 2.0 * (2 * (double)M * C + 2 * elements_w + 2 * elements_x) / 5e6;
        double time = c.base + (end > reads ? end : reads);
        if (px > 1 || pw > 1)
          time += c.join + 0.15 * (px > pw ? px : pw) + c.join_sum * 1e-6 * ((px > 1 ? px * elements_x : 0) + (pw > 1 ? pw * elements_w : 0));
        if (time < least) *best = {body, px, pw, dw_first}, least = time, found = true;
      }
    }
  }
  return found;
}
// One of them by itself: 128 x 128 tiles with as many pieces (all such bodies add a piece's products in the same order), so that
// its values do not depend on whether the other is asked for. Over 37 sizes dx takes 5% longer for it than with its own best body
// and pieces (512 x 1024 x 1024: 12.8 us for 10.1 with tiles of 64 x 128, the worst), dw 1% (11% at worst).
Plan one_of(int64_t rows, int64_t columns, int64_t sum, int pieces) {
  const double one = tile_time(dense::kTile128, rows, columns, sum, pieces), two = tile_time(dense::kTile128Pair, rows, columns, sum, pieces);
  return {one < two ? (int)dense::kTile128 : (int)dense::kTile128Pair, pieces, one < two ? one : two};
}

bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }

// A matrix as an operand: rows at 16-byte addresses whose last chunk of eight may be read, or a copy that has them.
struct Operand {
  const uint16_t* p;
  int64_t ld;
  int64_t half = 0; // elements from a row's first half to its second
};
bool direct(const void* p, int64_t ld, int64_t cols) {
  return aligned16(p) && ld % 8 == 0 && cols % 8 == 0 && ld <= kMaxDirectStride;
}

struct Call {
  pgemm_ctx* h; // null: only the scratch is counted
  dense::Kernels kernels;
  Scratch scratch;
  hipError_t status = hipSuccess;

  template <class K, class... A>
  void launch(int64_t grid, int threads, K kernel, A... args) {
    if (h && status == hipSuccess && grid > 0) status = enqueue(h->stream, dim3((unsigned)grid), dim3(threads), kernel, args...);
  }

  dense::SideArgs side = {}; // launched by prepare()
  int pads = 0;

  // wide: the rows can be used as they are; otherwise they are moved by prepare().
  Operand operand(const void* p, int64_t ld, int64_t rows, int64_t cols, int halves, bool wide) {
    Operand o = {static_cast<const uint16_t*>(p), ld, cols};
    if (wide) return o;
    const int64_t padded = round8(cols), chunks = padded / 8 * halves;
    uint16_t* to = scratch.take<uint16_t>(rows * padded * halves);
    side.pad[pads] = {o.p, ld, to, (int)rows, (int)cols, halves, (int)(padded / 8)};
    side.pad_blocks[pads++] = (int)((rows * chunks + 255) / 256);
    return {to, padded * halves, padded};
  }
  void prepare() {
    launch((int64_t)side.pad_blocks[0] + side.pad_blocks[1] + (side.C + 63) / 64, 256, kernels.side, side);
  }

  // The pieces' sums, and the tiles.
  void lay_out(Args& a, int body, int pieces, bool gated) {
    a.split = pieces;
    if (pieces > 1) a.part = scratch.take<float>(pieces * (int64_t)a.M * dense::part_ld(a, gated));
    const Tile t = tile_of(body);
    a.n_m = (int)((a.M + t.bm - 1) / t.bm);
    a.n_n = (int)(((gated ? 2 * (int64_t)a.N : a.N) + t.bn - 1) / t.bn);
  }
  static int64_t tile_groups(const Args& a) { return ((int64_t)a.n_m * a.n_n * a.split + 7) / 8 * 8; }
  static int64_t join_groups(const Args& a) { return a.split > 1 ? ((int64_t)a.M * ((a.N + 7) / 8) + 255) / 256 : 0; }

  void both(Args dx, Args dw, const Both& plan, int form) {
    lay_out(dx, plan.body, plan.split_x, false);
    lay_out(dw, plan.body, plan.split_w, false);
    if (!h) return;
    launch(tile_groups(dx) + tile_groups(dw), 512, kernels.pick_both(plan.body, form), dx, dw,
           (int)tile_groups(plan.dw_first ? dw : dx), (int)plan.dw_first);
    launch(join_groups(dx) + join_groups(dw), 256, kernels.join_both, dx, dw, (int)join_groups(dx));
  }

  void product(Args a, Plan plan, int form, bool gated) {
    lay_out(a, plan.body, plan.split, gated);
    if (!h) return;
    const dense::kernel_fn kernel = kernels.pick(plan.body, form, gated);
    if (plan.body <= dense::kFew32) {
      const int rows = few_rows(plan.body), wide = few_columns(form == dense::kRowsNK);
      if (status == hipSuccess)
        status = enqueue(h->stream, dim3((unsigned)((a.N + wide - 1) / wide), (unsigned)((a.M + rows - 1) / rows)), dim3(512), kernel, a);
      return;
    }
    const int64_t total = (int64_t)a.n_m * a.n_n * a.split;
    launch(plan.body != dense::kPing ? tile_groups(a) : total < h->cus ? total : h->cus, 512, kernel, a);
    launch(join_groups(a), 256, kernels.join[gated], a);
  }
};

int check(pgemm_ctx* h, int64_t M, int64_t N, int64_t K, int layout, int act, int gated, int dtype) {
  if (M < 0 || N < 0 || K < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "sizes M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (layout != PGEMM_B_KN && layout != PGEMM_B_NK) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown layout %d", layout);
  if (act < 0 || act >= act::kActs) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown activation %d", act);
  if (gated != 0 && gated != 1) return fail(h, PGEMM_ERR_INVALID_ARG, "gated is %d, not 0 or 1", gated);
  if (dtype != PGEMM_F16 && dtype != PGEMM_BF16) return fail(h, PGEMM_ERR_INVALID_ARG, "dtype %d is not fp16 or bf16", dtype);
  if (M > kMaxSize || N > kMaxSize || K > kMaxSize) return fail(h, PGEMM_ERR_UNSUPPORTED, "sizes must not exceed 2^30");
  // 2^21 tiles of 64 x 128, 512 threads each, where a launch takes 2^32 threads (more pieces than one only up to 1024
  // workgroups); rows that a tile's offsets span
  const int64_t C = gated ? 2 * N : N;
  auto tiles = [](int64_t a, int64_t b) { return ((a + 63) / 64) * ((b + 127) / 128); };
  if (tiles(M, C) > (1 << 21) || tiles(M, K) > (1 << 21) || tiles(C, K) > (1 << 21) || C > kMaxDirectStride || K > kMaxDirectStride)
    return fail(h, PGEMM_ERR_UNSUPPORTED, "M=%lld N=%lld K=%lld are more than one launch takes", (long long)M, (long long)N, (long long)K);
  return PGEMM_OK;
}

int forward(Call& c, const void* x, int64_t ldx, const void* w, int64_t ldw, bool wide_x, bool wide_w, Args a, int layout, bool gated) {
  const bool nk = layout == PGEMM_B_NK;
  const int form = nk ? dense::kRowsNK : dense::kRowsKN;
  const Plan plan = plan_rows(a.M, a.N, a.K, nk, gated, a.K % 8, (nk ? a.K : a.N) % 8);
  const int64_t columns = gated ? 2 * (int64_t)a.N : a.N;
  if (plan.body <= dense::kFew32) {
    a.a = static_cast<const uint16_t*>(x);
    a.lda = ldx;
    a.b = static_cast<const uint16_t*>(w);
    a.ldb = ldw;
    a.half = nk ? a.N * ldw : a.N;
  } else {
    const Operand xo = c.operand(x, ldx, a.M, a.K, 1, wide_x);
    const Operand wo = nk ? c.operand(w, ldw, columns, a.K, 1, wide_w) : c.operand(w, ldw, a.K, a.N, gated ? 2 : 1, wide_w);
    a.a = xo.p;
    a.lda = xo.ld;
    a.b = wo.p;
    a.ldb = wo.ld;
    a.half = nk ? a.N * wo.ld : wo.half;
    c.prepare();
  }
  c.product(a, plan, form, gated);
  return PGEMM_OK;
}

// Stretches of the rows whose column sums are formed separately: enough workgroups to fill the card, 16 rows each at least.
int stretches_of(int64_t M, int64_t N) {
  const int64_t blocks = (N + 511) / 512;
  int64_t s = 1024 / (blocks > 0 ? blocks : 1), most = (M + 15) / 16;
  if (s < 1) s = 1;
  if (s > most) s = most > 0 ? most : 1;
  return (int)(s > 512 ? 512 : s);
}

struct Gradients {
  const void *dy, *x, *w, *z;
  int64_t lddy, ldx, ldw;
  void *dx, *dw, *db;
  int64_t M, N, K;
  int layout, act;
  bool gated;
  bool wide_dy, wide_x, wide_w; // whether the rows can be used as they are
  bool need_dx, need_dw, need_db;
};

void backward(Call& c, const Gradients& g) {
  const int64_t C = g.gated ? 2 * g.N : g.N;
  const bool nk = g.layout == PGEMM_B_NK, slope = g.act != act::kNone || g.gated;
  const bool products = (g.need_dx || g.need_dw) && g.K > 0;
  Operand dz = {static_cast<const uint16_t*>(g.dy), g.lddy};
  const bool write = products && (slope || !g.wide_dy);
  if (write || g.need_db) {
    dense::ActGradArgs a = {};
    a.dy = dz.p;
    a.lddy = g.lddy;
    a.z = slope ? static_cast<const uint16_t*>(g.z) : nullptr;
    a.lddz = round8(C);
    if (write) {
      a.dz = c.scratch.take<uint16_t>(g.M * a.lddz);
      dz = {a.dz, a.lddz};
    }
    a.M = (int)g.M;
    a.N = (int)g.N;
    a.act = g.act;
    a.stretches = stretches_of(g.M, g.N);
    a.stream = g.N % 8 == 0 && 2 * g.M * (g.N + 2 * C) > (int64_t)256 << 20; // with dz, more than the cache's 256 MiB
    a.db = static_cast<uint16_t*>(g.db);
    if (g.need_db) a.part = c.scratch.take<float>(a.stretches * C);
    if (c.h && c.status == hipSuccess && g.N > 0)
      c.status = enqueue(c.h->stream, dim3((unsigned)((g.N + 511) / 512), (unsigned)a.stretches), dim3(256), c.kernels.act_grad[g.gated], a);
    if (g.need_db) {
      c.side.sums = a;
      c.side.C = (int)C;
    }
  }
  // dx = dz [M, C] times W, the sum running over W's columns; dW = x^T dz or its transpose
  const int form = nk ? dense::kRowsKN : dense::kRowsNK;
  Plan plan = plan_rows(g.M, g.K, C, !nk, false, false, (nk ? g.K : C) % 8);
  Operand w = {static_cast<const uint16_t*>(g.w), g.ldw}, x = {static_cast<const uint16_t*>(g.x), g.ldx};
  if (products && g.need_dx && plan.body > dense::kFew32)
    w = nk ? c.operand(g.w, g.ldw, C, g.K, 1, g.wide_w) : c.operand(g.w, g.ldw, g.K, C, 1, g.wide_w);
  if (products && g.need_dw) x = c.operand(g.x, g.ldx, g.M, g.K, 1, g.wide_x);
  c.prepare();
  if (!products) return;
  Args dx = {}, dw = {};
  dx.a = dz.p;
  dx.lda = dz.ld;
  dx.b = w.p;
  dx.ldb = w.ld;
  dx.c = static_cast<uint16_t*>(g.dx);
  dx.M = (int)g.M;
  dx.N = (int)g.K;
  dx.K = (int)C;
  dw.a = nk ? dz.p : x.p;
  dw.lda = nk ? dz.ld : x.ld;
  dw.b = nk ? x.p : dz.p;
  dw.ldb = nk ? x.ld : dz.ld;
  dw.c = static_cast<uint16_t*>(g.dw);
  dw.M = (int)(nk ? C : g.K);
  dw.N = (int)(nk ? g.K : C);
  dw.K = (int)g.M;
  Plan dw_plan = plan_grad(g.M, dw.M, dw.N);
  Both both;
  if (plan_both(g.M, g.K, C, nk, plan, dw_plan, &both)) {
    if (g.need_dx && g.need_dw) return c.both(dx, dw, both, form);
    plan = one_of(g.M, g.K, C, both.split_x); // the same sums, to the bit, where one of them is wanted
    dw_plan = one_of(dw.M, dw.N, g.M, both.split_w);
  }
  if (g.need_dx) c.product(dx, plan, form, false);
  if (g.need_dw) c.product(dw, dw_plan, dense::kGrad, false);
}

int short_of(pgemm_ctx* h, int64_t need, const void* work, int64_t have) {
  if (have < need || (need && (!work || !aligned16(work))))
    return fail(h, PGEMM_ERR_INVALID_ARG, "workspace of %lld bytes at %p, %lld at a multiple of 16 are needed", (long long)have, work,
                (long long)need);
  return PGEMM_OK;
}

dense::Kernels kernels_of(int dtype) { return dtype == PGEMM_F16 ? dense::kernels_f16() : dense::kernels_bf16(); }

} // namespace

extern "C" {

int pgemm_dense_workspace(int64_t M, int64_t N, int64_t K, int layout, int gated, int wide, int64_t* bytes) {
  if (!bytes) return PGEMM_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = check(nullptr, M, N, K, layout, 0, gated, PGEMM_F16);
  if (rc != PGEMM_OK || M == 0 || N == 0) return rc;
  Call c = {nullptr, {}, {nullptr}};
  Args a = {};
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  const bool kn = layout == PGEMM_B_KN;
  forward(c, nullptr, K, nullptr, 0, wide && K % 8 == 0, wide && (kn ? N : K) % 8 == 0, a, layout, gated);
  *bytes = c.scratch.used;
  return PGEMM_OK;
}

int pgemm_dense_run(pgemm_handle_t h, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                    const void* residual, int64_t ldr, void* y, void* z, int64_t M, int64_t N, int64_t K, int layout, int act,
                    int gated, int dtype, void* work, int64_t work_bytes) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  int rc = check(h, M, N, K, layout, act, gated, dtype);
  if (rc != PGEMM_OK) return rc;
  const bool nk = layout == PGEMM_B_NK;
  if (ldx < 0 || ldr < 0 || ldw < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "row strides %lld, %lld, %lld", (long long)ldx, (long long)ldw, (long long)ldr);
  if (M == 0 || N == 0) return PGEMM_OK;
  if (!y || (K > 0 && (!x || !w))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  Args a = {};
  a.bias = static_cast<const uint16_t*>(bias);
  a.residual = static_cast<const uint16_t*>(residual);
  a.ldr = ldr;
  a.c = static_cast<uint16_t*>(y);
  a.z = static_cast<uint16_t*>(z);
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.act = act;
  const bool wide_x = direct(x, ldx, K), wide_w = direct(w, ldw, nk ? K : N);
  Call count = {nullptr, {}, {nullptr}};
  forward(count, x, ldx, w, ldw, wide_x, wide_w, a, layout, gated);
  rc = short_of(h, count.scratch.used, work, work_bytes);
  if (rc != PGEMM_OK) return rc;
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  Call c = {h, kernels_of(dtype), {static_cast<char*>(work)}};
  forward(c, x, ldx, w, ldw, wide_x, wide_w, a, layout, gated);
  return launch_status(h, c.status, "linear layer");
}

int pgemm_dense_backward_workspace(int64_t M, int64_t N, int64_t K, int layout, int act, int gated, int needs, int wide,
                                   int64_t* bytes) {
  if (!bytes || needs < 0 || needs > 7) return PGEMM_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = check(nullptr, M, N, K, layout, act, gated, PGEMM_F16);
  if (rc != PGEMM_OK) return rc;
  Call c = {nullptr, {}, {nullptr}};
  Gradients g = {};
  g.M = M;
  g.N = N;
  g.K = K;
  g.layout = layout;
  g.act = act;
  g.gated = gated;
  const int64_t columns = gated ? 2 * N : N;
  g.wide_dy = wide && N % 8 == 0;
  g.wide_x = wide && K % 8 == 0;
  g.wide_w = wide && (layout == PGEMM_B_NK ? K : columns) % 8 == 0;
  g.need_dx = needs & PGEMM_DENSE_DX;
  g.need_dw = needs & PGEMM_DENSE_DW;
  g.need_db = needs & PGEMM_DENSE_DB;
  backward(c, g);
  *bytes = c.scratch.used;
  return PGEMM_OK;
}

int pgemm_dense_backward(pgemm_handle_t h, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                         const void* z, void* dx, void* dw, void* db, int64_t M, int64_t N, int64_t K, int layout, int act,
                         int gated, int dtype, void* work, int64_t work_bytes) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  int rc = check(h, M, N, K, layout, act, gated, dtype);
  if (rc != PGEMM_OK) return rc;
  if (lddy < 0 || ldx < 0 || ldw < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "row strides %lld, %lld, %lld", (long long)lddy, (long long)ldx, (long long)ldw);
  const bool slope = act != act::kNone || gated, sums = M > 0 && N > 0;
  if (sums && (dx || dw || db) && (!dy || (slope && !z))) return fail(h, PGEMM_ERR_INVALID_ARG, "dy or z is NULL");
  if (sums && K > 0 && ((dx && !w) || (dw && !x))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  const int64_t columns = gated ? 2 * N : N;
  Gradients g = {dy, x, w, z, lddy, ldx, ldw, dx, dw, db, M, N, K, layout, act, gated != 0};
  g.wide_dy = direct(dy, lddy, N);
  g.wide_x = direct(x, ldx, K);
  g.wide_w = direct(w, ldw, layout == PGEMM_B_NK ? K : columns);
  g.need_dx = dx && M > 0;
  g.need_dw = dw && N > 0;
  g.need_db = db && N > 0;
  Call count = {nullptr, {}, {nullptr}};
  backward(count, g);
  rc = short_of(h, count.scratch.used, work, work_bytes);
  if (rc != PGEMM_OK) return rc;
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  Call c = {h, kernels_of(dtype), {static_cast<char*>(work)}};
  backward(c, g);
  return launch_status(h, c.status, "linear layer's gradient");
}

int pgemm_dense_query(int64_t M, int64_t N, int64_t K, int layout, int gated, int* body, int* pieces) {
  if (!body || !pieces || M < 1 || N < 1 || K < 1) return PGEMM_ERR_INVALID_ARG;
  const int rc = check(nullptr, M, N, K, layout, 0, gated, PGEMM_F16);
  if (rc != PGEMM_OK) return rc;
  const bool nk = layout == PGEMM_B_NK;
  const Plan p = plan_rows(M, N, K, nk, gated, K % 8, (nk ? K : N) % 8);
  *body = p.body;
  *pieces = p.split;
  return PGEMM_OK;
}

int pgemm_dense_weight_grad_query(int64_t R, int64_t I, int64_t J, int* body, int* pieces) {
  if (!body || !pieces || R < 1 || I < 1 || J < 1) return PGEMM_ERR_INVALID_ARG;
  const int rc = check(nullptr, R, I, J, PGEMM_B_NK, 0, 0, PGEMM_F16);
  if (rc != PGEMM_OK) return rc;
  const Plan p = plan_grad(R, I, J);
  *body = p.body;
  *pieces = p.split;
  return PGEMM_OK;
}

int pgemm_dense_gradients_query(int64_t M, int64_t C, int64_t K, int layout, int* body, int* pieces_dx, int* pieces_dw) {
  if (!body || !pieces_dx || !pieces_dw || M < 1 || C < 1 || K < 1) return PGEMM_ERR_INVALID_ARG;
  const int rc = check(nullptr, M, C, K, layout, 0, 0, PGEMM_F16);
  if (rc != PGEMM_OK) return rc;
  const bool nk = layout == PGEMM_B_NK;
  const Plan dx = plan_rows(M, K, C, !nk, false, false, (nk ? K : C) % 8), dw = plan_grad(M, nk ? C : K, nk ? K : C);
  Both both;
  const bool one = plan_both(M, K, C, nk, dx, dw, &both);
  *body = one ? both.body : -1;
  *pieces_dx = one ? both.split_x : dx.split;
  *pieces_dw = one ? both.split_w : dw.split;
  return PGEMM_OK;
}

} // extern "C"
