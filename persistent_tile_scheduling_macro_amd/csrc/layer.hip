// Entry point of the routed layer of few tokens.
#include "context.h"
#include "layer.h"

using namespace pgemm;

namespace {

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// Blocks of 16 rows in a group, by the mean number of tokens that take an awake expert (n slots among E experts leave
// E (1 - 1/E)^n of them asleep): up to 6 rows rarely exceed 16, up to 16 rarely 32.
int blocks_of(int64_t T, int64_t k, int64_t E) {
  const double n = (double)T * k, mean = n / (E * (1 - __builtin_exp(-n / E)));
  if (T <= 16 || mean <= 6) return 1;
  return T <= 32 || mean <= 16 ? 2 : 4;
}

// Workspace of a pass of T tokens.
struct Parts { int64_t slots, shares, arrived, parts, h, bytes, most, sharers; };
Parts parts_of(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int cus) {
  const int64_t t = T < layer::kTokens ? T : layer::kTokens, n = t * k, tiles = (H + 15) / 16;
  const int blocks = blocks_of(t, k, E);
  Parts p = {};
  p.most = (E < n ? E : n) + n / (16 * blocks); // whole groups and each expert's last
  const int64_t room = (E < n ? E : n) + n / 16; // a last pass of fewer tokens may have smaller groups, and more of them
  // Workgroups that share 16 columns of out: enough for every CU, each wave with two steps at least.
  const int64_t steps = p.most * ((I + 63) / 64), fill = tiles > 0 ? cus / tiles : 1, long_enough = steps / (2 * layer::down_waves(blocks));
  p.sharers = fill < long_enough ? fill : long_enough;
  p.sharers = p.sharers < 1 ? 1 : p.sharers > 16 ? 16 : p.sharers;
  p.slots = round256((room + 1) * 4);
  p.shares = p.slots + round256(room * layer::kTokens * 4);
  p.arrived = p.shares + round256(room * layer::kTokens * 4);
  p.parts = p.arrived + round256(tiles * 4);
  p.h = p.parts + round256(tiles * p.sharers * t * 64);
  p.bytes = p.h + round256(n * I * 2);
  return p;
}
constexpr int kCus = 256; // the workspace is the same whatever device runs it

int check(pgemm_ctx* h, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  if (T < 0 || k < 1 || E < 1 || H < 0 || I < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "sizes T=%lld k=%lld E=%lld H=%lld I=%lld", (long long)T, (long long)k, (long long)E,
                (long long)H, (long long)I);
  if (E > moe::kMaxExperts || k > layer::kMaxSlots / layer::kTokens || T > 4096 || H > (int64_t)1 << 20 || I > (int64_t)1 << 19)
    return fail(h, PGEMM_ERR_UNSUPPORTED,
                "T=%lld k=%lld E=%lld H=%lld I=%lld: at most 4096 tokens, %d choices, %d experts, rows of 2^20 and 2^19", (long long)T,
                (long long)k, (long long)E, (long long)H, (long long)I, layer::kMaxSlots / layer::kTokens, moe::kMaxExperts);
  return PGEMM_OK;
}

} // namespace

extern "C" {

int pgemm_moe_layer_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t* bytes) {
  if (!bytes) return PGEMM_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = check(nullptr, T, k, E, H, I);
  if (rc == PGEMM_OK && T > 0) *bytes = parts_of(T, k, E, H, I, kCus).bytes;
  return rc;
}

int pgemm_moe_layer(pgemm_handle_t h, const void* x, int64_t ldx, const void* ids, int ids_type, const float* weights,
                    const void* w_in, const void* w_out, void* out, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int act,
                    int gated, int dtype, void* work, int64_t work_bytes) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  const int rc = check(h, T, k, E, H, I);
  if (rc != PGEMM_OK) return rc;
  if (ldx < 0) return fail(h, PGEMM_ERR_INVALID_ARG, "row stride %lld", (long long)ldx);
  if (ids_type != PGEMM_IDS_I32 && ids_type != PGEMM_IDS_I64) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown type of ids %d", ids_type);
  if (act < 0 || act >= act::kActs) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown activation %d", act);
  if (gated != 0 && gated != 1) return fail(h, PGEMM_ERR_INVALID_ARG, "gated is %d, not 0 or 1", gated);
  if (dtype != PGEMM_F16 && dtype != PGEMM_BF16) return fail(h, PGEMM_ERR_INVALID_ARG, "dtype %d is not fp16 or bf16", dtype);
  if (T == 0 || H == 0) return PGEMM_OK;
  if (!x || !ids || !weights || !out || (I > 0 && (!w_in || !w_out))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  const Parts p = parts_of(T, k, E, H, I, kCus);
  if (!work || work_bytes < p.bytes || (uintptr_t)work % 16)
    return fail(h, PGEMM_ERR_INVALID_ARG, "workspace of %lld bytes at %p, %lld at a multiple of 16 are needed", (long long)work_bytes,
                work, (long long)p.bytes);
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  if (I == 0) return launch_status(h, launch_fill_zero(out, T, H, H, h->stream), "zero-fill"); // empty sums
  char* base = static_cast<char*>(work);
  layer::Args a = {};
  a.ldx = ldx;
  a.ids64 = ids_type == PGEMM_IDS_I64;
  a.w_in = static_cast<const uint16_t*>(w_in);
  a.w_out = static_cast<const uint16_t*>(w_out);
  a.h = reinterpret_cast<uint16_t*>(base + p.h);
  a.groups = reinterpret_cast<int*>(base);
  a.slots = reinterpret_cast<int*>(base + p.slots);
  a.shares = reinterpret_cast<float*>(base + p.shares);
  a.arrived = reinterpret_cast<int*>(base + p.arrived);
  a.parts = reinterpret_cast<float*>(base + p.parts);
  a.k = (int)k;
  a.E = (int)E;
  a.H = (int)H;
  a.I = (int)I;
  a.act = act;
  const bool f16 = dtype == PGEMM_F16;
  hipError_t e = hipSuccess;
  for (int64_t t = 0; e == hipSuccess && t < T; t += layer::kTokens) { // more tokens than one pass has: each reads the matrices again
    a.T = (int)(T - t < layer::kTokens ? T - t : layer::kTokens);
    a.x = static_cast<const uint16_t*>(x) + t * ldx;
    a.ids = static_cast<const char*>(ids) + t * k * (a.ids64 ? 8 : 4);
    a.weights = weights + t * k;
    a.out = static_cast<uint16_t*>(out) + t * H;
    const Parts q = parts_of(a.T, k, E, H, I, kCus); // laid out like the first pass
    const int blocks = blocks_of(a.T, k, E);
    a.most = (int)q.most;
    a.sharers = (int)(q.sharers < p.sharers ? q.sharers : p.sharers);
    const int64_t tiles = (I + 15) / 16, fill = (512 + a.most - 1) / a.most; // two workgroups a CU
    // Several turns of columns a workgroup for short rows. Measured at 45 sizes (profiles/dense_layer_rules.txt): up to H = 1024
    // one turn each is from 14% faster to 40% slower, 4% slower in the mean; past it several are from 2% faster to 21% slower.
    const bool loop = H <= 1024 && fill < tiles;
    e = enqueue(h->stream, dim3((unsigned)(loop ? fill : tiles), (unsigned)a.most), dim3(512),
                f16 ? layer::up_f16(gated, blocks, loop) : layer::up_bf16(gated, blocks, loop), a);
    if (e == hipSuccess)
      e = enqueue(h->stream, dim3((unsigned)((H + 15) / 16), (unsigned)a.sharers), dim3(64 * layer::down_waves(blocks)),
                  f16 ? layer::down_f16(blocks, I < 8) : layer::down_bf16(blocks, I < 8), a);
  }
  return launch_status(h, e, "routed layer");
}

} // extern "C"
