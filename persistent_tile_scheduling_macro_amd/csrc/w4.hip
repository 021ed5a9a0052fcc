// Entry point of the product with 4-bit weights.
#include "context.h"
#include "w4.h"

using namespace pgemm;

namespace {

struct Form { int rows, blocks; };
Form pick_form(int64_t M, int64_t N, int64_t E, bool offsets, int cus) {
  // Rows a workgroup takes at once. An expert's rows are known only on the device: twice the mean
  // covers most experts in one pass, and a longer one loops.
  const int64_t mean = offsets ? (2 * M + E - 1) / E : M;
  // Columns a wave takes: two blocks share the reads of x, one where two would leave CUs idle.
  const int64_t experts = offsets ? (E < M ? E : M) : 1;
  return {mean <= 4 ? 4 : mean <= 16 ? 16 : 32, experts * ((N + 31) / 32) >= 2 * cus ? 2 : 1};
}

} // namespace

extern "C" int pgemm_w4_query(int64_t M, int64_t N, int64_t E, int experts, int cus, int* rows, int* blocks) {
  if (!rows || !blocks || M < 1 || N < 1 || E < 1 || cus < 1) return PGEMM_ERR_INVALID_ARG;
  constexpr int64_t lim = (int64_t)1 << 30;
  if (M > lim || N > lim || E > 65534) return PGEMM_ERR_UNSUPPORTED;
  const Form f = pick_form(M, N, E, experts != 0, cus);
  *rows = f.rows;
  *blocks = f.blocks;
  return PGEMM_OK;
}

extern "C" int pgemm_w4_run(pgemm_handle_t h, const void* x, int64_t ldx, const void* q, const void* scales,
                            const void* zeros, const int32_t* offsets, void* y, int64_t M, int64_t N, int64_t K,
                            int64_t E, int group, int fmt, int dtype) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  if (M < 0 || N < 0 || K < 0 || E < 1 || ldx < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "sizes M=%lld N=%lld K=%lld E=%lld ldx=%lld", (long long)M, (long long)N,
                (long long)K, (long long)E, (long long)ldx);
  if (group != 32 && group != 64 && group != 128)
    return fail(h, PGEMM_ERR_INVALID_ARG, "group of %d, not 32, 64 or 128", group);
  if (fmt != PGEMM_W4_INT4 && fmt != PGEMM_W4_E2M1) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown 4-bit format %d", fmt);
  if (dtype != PGEMM_F16 && dtype != PGEMM_BF16)
    return fail(h, PGEMM_ERR_INVALID_ARG, "dtype %d is not fp16 or bf16", dtype);
  if (zeros && fmt != PGEMM_W4_INT4) return fail(h, PGEMM_ERR_INVALID_ARG, "e2m1 weights have no zero points");
  if (!offsets && E != 1) return fail(h, PGEMM_ERR_INVALID_ARG, "E=%lld experts without offsets", (long long)E);
  constexpr int64_t lim = (int64_t)1 << 30;
  if (M > lim || N > lim || K > lim) return fail(h, PGEMM_ERR_UNSUPPORTED, "sizes must not exceed 2^30");
  if (E > 65534) return fail(h, PGEMM_ERR_UNSUPPORTED, "E=%lld experts, at most 65534", (long long)E);
  if (M == 0 || N == 0) return PGEMM_OK;
  if (!y || (K > 0 && (!x || !q || !scales))) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  if (K == 0) { // an empty sum
    return launch_status(h, launch_fill_zero(y, M, N, N, h->stream), "zero-fill");
  }
  w4::Args a;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.q = static_cast<const uint8_t*>(q);
  a.scales = static_cast<const uint16_t*>(scales);
  a.zeros = static_cast<const uint8_t*>(zeros);
  a.offsets = offsets;
  a.y = static_cast<uint16_t*>(y);
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.E = (int)E;
  a.row_bytes = (int)((K + 1) / 2);
  a.groups = (int)((K + group - 1) / group);
  const auto [rows, cb] = pick_form(M, N, E, offsets != nullptr, h->cus);
  const int64_t row_groups = offsets ? E + 1 : (M + rows - 1) / rows;
  const int64_t cols = (N + 16 * cb - 1) / (16 * cb);
  if (cols * w4::waves_of(rows) * 64 > UINT32_MAX) // threads of a launch
    return fail(h, PGEMM_ERR_UNSUPPORTED, "N=%lld columns are more than one launch takes", (long long)N);
  const int form = zeros ? w4::kInt4Zero : fmt == PGEMM_W4_E2M1 ? w4::kE2M1 : w4::kInt4;
  const w4::kernel_fn kern = dtype == PGEMM_F16 ? w4::pick_f16(form, group, rows, cb) : w4::pick_bf16(form, group, rows, cb);
  if (row_groups <= 65535) {
    return launch_status(h, enqueue(h->stream, dim3((unsigned)cols, (unsigned)row_groups), dim3(w4::waves_of(rows) * 64), kern, a),
                         "w4");
  }
  // more rows than one grid has: launches of at most 65535 row groups each
  hipError_t e = hipSuccess;
  for (int64_t r = 0; e == hipSuccess && r < row_groups; r += 65535) {
    w4::Args b = a;
    const int64_t from = r * rows, count = row_groups - r < 65535 ? row_groups - r : 65535;
    b.x = a.x + from * ldx;
    b.y = a.y + from * N;
    b.M = (int)(M - from < count * rows ? M - from : count * rows);
    e = enqueue(h->stream, dim3((unsigned)cols, (unsigned)count), dim3(w4::waves_of(rows) * 64), kern, b);
  }
  return launch_status(h, e, "w4");
}
