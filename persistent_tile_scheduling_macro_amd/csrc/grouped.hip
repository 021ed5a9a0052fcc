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

int launch(pgemm_ctx* h, const grouped::Args& a, int64_t tiles, int dtype, bool grad, bool nk) {
  if (tiles > INT32_MAX - 8) return fail(h, PGEMM_ERR_UNSUPPORTED, "more than 2^31 output tiles");
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  const grouped::kernel_fn kern = dtype == PGEMM_F16 ? grouped::pick_f16(grad, nk) : grouped::pick_bf16(grad, nk);
  hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(256), 0, h->stream, a);
  return launch_status(h, "grouped product");
}

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
  a.n_n = (int)((N + 127) / 128);
  // every expert, and the rows of none, may leave one tile partly filled; a multiple of 8 for the XCDs
  const int64_t tiles = ((R / 128 + E + 1) * a.n_n + 7) / 8 * 8;
  return launch(h, a, tiles, dtype, false, layout == PGEMM_B_NK);
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
  a.n_n = (int)((J + 127) / 128);
  return launch(h, a, E * ((I + 127) / 128) * a.n_n, dtype, true, false);
}

} // extern "C"
