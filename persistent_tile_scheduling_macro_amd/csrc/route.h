// The router: each token's k experts and their weights, from its logits.
//
// The largest k logits are chosen, the first of equal ones; -inf and NaN are
// never chosen (a token with fewer others gets the id -1 and the weight 0 in
// the places left, a dropped slot for dispatch). Scores:
//   softmax  s_e = exp(l_e - max) / sum_e exp(l_e - max)
//   sigmoid  s_e = 1 / (1 + exp(-l_e))
// weights: the chosen scores, normalized: over their sum. That sum is formed
// without underflow: of exp(l_e - max) for the softmax, and for sigmoids whose
// largest logit is negative of exp(l_e - max) / (1 + exp(l_e)), the same
// multiple of each. Gradients, with d the weights' and D = sum w d:
//   softmax     dl = s (d - D) over all experts, d = 0 where not chosen
//   sigmoid     dl = d s (1 - s) on the chosen
//   normalized  dl = w (d - D), for the sigmoid times (1 - s), on the chosen
//
// A token's logits lie in registers: PER of them in each of LANES lanes, a
// whole wave or, for up to 32 experts, a part of one. A choice by a whole wave
// is a maximum over its lanes by DPP (the logits as ordered integers) and a
// ballot that finds the first lane that has it; a part of a wave takes a
// butterfly over a 64-bit key instead (the integer, then the expert,
// inverted). Lane c keeps choice c, so that all scores are one exponential.
// The bytes are few: the launch, then the instructions of the k choices bound it
// (8192 tokens, 8 of 256 experts: 8.1 us, with butterflies of the whole wave 14.5;
// the gradient 7.7; 16 tokens, 8 of 64: 3.2 us, a bare launch).
#pragma once

#include "moe_rows.h"

namespace pgemm {
namespace route {

constexpr int kThreads = 256;
constexpr int kMaxChoices = 64;
enum Type : int { kF16 = 0, kBF16 = 1, kF32 = 3 };
enum Score : int { kSoftmax = 0, kSigmoid = 1 };

struct Args {
  const void* logits; // T rows, ld apart
  int64_t ld;
  int* ids;              // [T, k]
  float* weights;        // [T, k]
  const float* dweights; // backward: [T, k]
  void* dlogits;         // backward: [T, E]
  int T, E, k, score, normalize;
};

// A logit; NaN is what -inf is.
template <int TY>
__device__ inline float load(const void* p, int64_t i) {
  float v;
  if constexpr (TY == kF32) v = static_cast<const float*>(p)[i];
  else if constexpr (TY == kBF16) v = __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else v = (float)static_cast<const _Float16*>(p)[i];
  return v == v ? v : -__builtin_huge_valf();
}
template <int TY>
__device__ inline void store(void* p, int64_t i, float v) {
  if constexpr (TY == kF32) static_cast<float*>(p)[i] = v;
  else if constexpr (TY == kBF16) static_cast<__bf16*>(p)[i] = (__bf16)v;
  else static_cast<_Float16*>(p)[i] = (_Float16)v;
}

// Logits in order as unsigned numbers; 0 for what is never chosen.
__device__ inline uint32_t order_of(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f); // -0 is 0
  return l == -__builtin_huge_valf() ? 0 : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline float logit_of(uint32_t o) { return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }

template <int LANES>
__device__ inline float sum_lanes(float v) {
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Largest of a whole wave's values, in every lane (all 64 take part).
__device__ inline uint32_t wave_max(uint32_t v) {
#define PGEMM_DPP_MAX(CTRL, ROWS) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false))
  PGEMM_DPP_MAX(0x111, 0xF); // row_shr 1, 2, 4, 8: lane 15 of each row has the row's
  PGEMM_DPP_MAX(0x112, 0xF);
  PGEMM_DPP_MAX(0x114, 0xF);
  PGEMM_DPP_MAX(0x118, 0xF);
  PGEMM_DPP_MAX(0x142, 0xA); // row_bcast 15 into rows 1 and 3, row_bcast 31 into rows 2 and 3
  PGEMM_DPP_MAX(0x143, 0xC);
#undef PGEMM_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// exp and 1 / x by the hardware's exp2 and reciprocal, each off by a step; x log2(e) adds |x| 2^-24 to exp's relative error.
// (With the library's the kernels took 8.8 and 9.4 us instead of 8.1 and 7.7: instructions bound them.)
__device__ inline float fast_exp(float x) { return __builtin_amdgcn_exp2f(1.44269504f * x); }
__device__ inline float inverse(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ inline float logistic(float l) { return inverse(1.0f + fast_exp(-l)); }

// k is at most LANES: lane c of a token keeps its choice c.
template <int TY, int LANES, int PER>
__global__ void __launch_bounds__(kThreads) choose_kernel(Args a) {
  const int lane = threadIdx.x % LANES;
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LANES;
  if (t >= a.T) return; // all of a token's lanes
  float l[PER];
  uint32_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + LANES * j;
    l[j] = e < a.E ? load<TY>(a.logits, t * a.ld + e) : -__builtin_huge_valf();
    key[j] = order_of(l[j]);
  }
  float logit = 0.0f;
  int id = -1;
  for (int c = 0; c < a.k; ++c) {
    uint32_t best = 0;
    int e;
    if constexpr (LANES == 64) {
#pragma unroll
      for (int j = 0; j < PER; ++j) best = max(best, key[j]);
      best = wave_max(best);
      e = 0;
#pragma unroll
      for (int j = PER - 1; j >= 0; --j) { // the first expert that has it
        const uint64_t has = __ballot(key[j] == best);
        if (has) e = 64 * j + (int)__builtin_ctzll(has);
      }
    } else {
      static_assert(PER == 1 || LANES == 64, "a part of a wave holds a logit a lane");
      uint64_t v = (uint64_t)key[0] << 32 | (uint32_t) ~lane;
#pragma unroll
      for (int d = LANES / 2; d; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d);
        if (o > v) v = o;
      }
      best = (uint32_t)(v >> 32);
      e = (int)~(uint32_t)v;
    }
    if (best == 0) break; // nothing is left for this token
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (lane + LANES * j == e) key[j] = 0;
    if (lane == c) {
      logit = logit_of(best);
      id = e;
    }
  }
  const float most = __shfl(logit, 0, LANES); // the first choice; 0 where there is none
  float score = 0.0f, total = 0.0f;
  if (id >= 0) {
    if (a.score == kSoftmax) score = fast_exp(logit - most);
    else score = a.normalize && most < 0.0f ? fast_exp(logit - most) * inverse(1.0f + fast_exp(logit)) : logistic(logit);
  }
  if (a.normalize) {
    total = score;
  } else if (a.score == kSoftmax) {
#pragma unroll
    for (int j = 0; j < PER; ++j) total += fast_exp(l[j] - most);
  }
  const float over = a.normalize || a.score == kSoftmax ? inverse(sum_lanes<LANES>(total)) : 1.0f;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.weights[t * a.k + lane] = id < 0 ? 0.0f : score * over;
  }
}

template <int TY, int LANES, int PER>
__global__ void __launch_bounds__(kThreads) choose_backward_kernel(Args a) {
  const int lane = threadIdx.x % LANES;
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LANES;
  if (t >= a.T) return;
  const bool all = a.score == kSoftmax && !a.normalize; // every expert has a part in the sum
  float l[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + LANES * j;
    l[j] = e < a.E ? load<TY>(a.logits, t * a.ld + e) : -__builtin_huge_valf();
  }
  int id = -1;
  float w = 0.0f, d = 0.0f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    if (id >= 0 && id < a.E) {
      w = a.weights[t * a.k + lane];
      d = a.dweights[t * a.k + lane];
    } else {
      id = -1;
    }
  }
  const float mean = sum_lanes<LANES>(w * d); // 0 where no choice was made
  // what its choice gives each of the lane's experts (choices that name one expert twice add up)
  const float gives = a.normalize ? w * (d - mean) : d;
  float part[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) part[j] = 0.0f;
  for (int c = 0; c < a.k; ++c) {
    int e;
    float p;
    if constexpr (LANES == 64) {
      e = __builtin_amdgcn_readlane(id, c);
      p = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, gives), c));
    } else {
      e = __shfl(id, c, LANES);
      p = __shfl(gives, c, LANES);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (lane + LANES * j == e) part[j] += p;
  }
  float over = 0.0f; // 1 / the softmax's sum
  if (all) {
    float most = -__builtin_huge_valf(), total = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) most = fmaxf(most, l[j]);
#pragma unroll
    for (int s = LANES / 2; s; s >>= 1) most = fmaxf(most, __shfl_xor(most, s));
    if (most == -__builtin_huge_valf()) most = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      l[j] = fast_exp(l[j] - most);
      total += l[j];
    }
    over = inverse(sum_lanes<LANES>(total));
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + LANES * j;
    if (e >= a.E) continue;
    float g = part[j];
    if (all) g = l[j] > 0.0f ? l[j] * over * (g - mean) : 0.0f;
    else if (a.score == kSigmoid) g *= a.normalize ? logistic(-l[j]) : logistic(l[j]) * logistic(-l[j]);
    store<TY>(a.dlogits, t * a.E + e, g);
  }
}

} // namespace route
} // namespace pgemm
