// Entry points of the router.
#include "context.h"
#include "route.h"

using namespace pgemm;

namespace {

static_assert((int)route::kSoftmax == (int)PGEMM_SCORE_SOFTMAX && (int)route::kSigmoid == (int)PGEMM_SCORE_SIGMOID,
              "the header's numbers are the scores'");
static_assert((int)route::kF16 == (int)PGEMM_LOGITS_F16 && (int)route::kBF16 == (int)PGEMM_LOGITS_BF16 &&
                  (int)route::kF32 == (int)PGEMM_LOGITS_F32,
              "the header's numbers are the types'");

typedef void (*kernel_fn)(route::Args);
struct Kernel { kernel_fn fn; int lanes; };

template <int TY>
Kernel pick(bool backward, int E) {
#define PGEMM_ROUTE(L, P) return {backward ? route::choose_backward_kernel<TY, L, P> : route::choose_kernel<TY, L, P>, L}
  if (E <= 8) PGEMM_ROUTE(8, 1);
  if (E <= 16) PGEMM_ROUTE(16, 1);
  if (E <= 32) PGEMM_ROUTE(32, 1);
  if (E <= 64) PGEMM_ROUTE(64, 1);
  if (E <= 128) PGEMM_ROUTE(64, 2);
  if (E <= 256) PGEMM_ROUTE(64, 4);
  if (E <= 512) PGEMM_ROUTE(64, 8);
  PGEMM_ROUTE(64, 16);
#undef PGEMM_ROUTE
}

int launch(pgemm_ctx* h, const route::Args& a, int type, bool backward) {
  const Kernel k = type == PGEMM_LOGITS_F32    ? pick<route::kF32>(backward, a.E)
                   : type == PGEMM_LOGITS_BF16 ? pick<route::kBF16>(backward, a.E)
                                               : pick<route::kF16>(backward, a.E);
  DeviceScope dev(h->device);
  if (!dev.ok()) return fail(h, PGEMM_ERR_HIP, "hipSetDevice failed");
  const int64_t per = route::kThreads / k.lanes;
  return launch_status(h, enqueue(h->stream, dim3((unsigned)((a.T + per - 1) / per)), dim3(route::kThreads), k.fn, a), "router");
}

int check(pgemm_ctx* h, int64_t ld, int64_t T, int64_t E, int64_t k, int score, int normalize, int type) {
  if (T < 0 || E < 1 || k < 1 || k > E || ld < 0)
    return fail(h, PGEMM_ERR_INVALID_ARG, "sizes T=%lld E=%lld k=%lld ld=%lld", (long long)T, (long long)E, (long long)k, (long long)ld);
  if (score != PGEMM_SCORE_SOFTMAX && score != PGEMM_SCORE_SIGMOID) return fail(h, PGEMM_ERR_INVALID_ARG, "unknown score %d", score);
  if (normalize != 0 && normalize != 1) return fail(h, PGEMM_ERR_INVALID_ARG, "normalize is %d, not 0 or 1", normalize);
  if (type != PGEMM_LOGITS_F16 && type != PGEMM_LOGITS_BF16 && type != PGEMM_LOGITS_F32)
    return fail(h, PGEMM_ERR_INVALID_ARG, "unknown type of logits %d", type);
  if (T > (int64_t)1 << 24 || E > moe::kMaxExperts || k > route::kMaxChoices)
    return fail(h, PGEMM_ERR_UNSUPPORTED, "T=%lld tokens, E=%lld experts, k=%lld choices: at most 2^24, %d, %d", (long long)T,
                (long long)E, (long long)k, moe::kMaxExperts, route::kMaxChoices);
  return PGEMM_OK;
}

} // namespace

extern "C" {

int pgemm_moe_route(pgemm_handle_t h, const void* logits, int64_t ld, int type, int64_t T, int64_t E, int64_t k, int score,
                    int normalize, int32_t* ids, float* weights) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  const int rc = check(h, ld, T, E, k, score, normalize, type);
  if (rc != PGEMM_OK || T == 0) return rc;
  if (!logits || !ids || !weights) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  return launch(h, {logits, ld, ids, weights, nullptr, nullptr, (int)T, (int)E, (int)k, score, normalize}, type, false);
}

int pgemm_moe_route_backward(pgemm_handle_t h, const float* dweights, const void* logits, int64_t ld, int type, const int32_t* ids,
                             const float* weights, int64_t T, int64_t E, int64_t k, int score, int normalize, void* dlogits) {
  if (!h) return PGEMM_ERR_INVALID_ARG;
  h->last_error[0] = 0;
  const int rc = check(h, ld, T, E, k, score, normalize, type);
  if (rc != PGEMM_OK || T == 0) return rc;
  if (!dweights || !logits || !ids || !weights || !dlogits) return fail(h, PGEMM_ERR_INVALID_ARG, "a pointer is NULL");
  return launch(h,
                {logits, ld, const_cast<int*>(ids), const_cast<float*>(weights), dweights, dlogits, (int)T, (int)E, (int)k, score,
                 normalize},
                type, true);
}

} // extern "C"
