// Activations of the linear layer and of the routed layer, in fp32.
//
//   relu       x below zero gives 0 (a NaN stays)
//   silu       x * s(x),                        s(u) = 1 / (1 + exp(-u))
//   gelu_tanh  x * (1 + tanh(r (x + 0.044715 x^3))) / 2 = x * s(2 r (x + 0.044715 x^3)),  r = sqrt(2 / pi)
//   gelu       x * Phi(x), Phi the normal distribution
// silu and gelu_tanh are one formula, x * s(x (c0 + c1 x^2)), with two
// constants. Phi needs the complementary error function with a small relative
// error, as its lower tail is the result: Phi(-a) = exp(-a^2 / 2) R(a), and R,
// which falls like 1/a, is a polynomial in t = 1 / (1 + 0.28 a), fitted to the
// function over all a >= 0 by weighted least squares, its relative error below
// 3.8e-6, a hundredth of half a step of fp16: some 16 instructions an element
// and no branch.
#pragma once

#include "device_common.h"

namespace pgemm {
namespace act {

enum Act : int { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4, kActs = 5 };
// The code paths: the activation is a launch's argument, so a kernel holds all three.
enum Path : int { kCopy, kLogistic, kNormal };

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Constants of one activation; uniform over a launch.
struct Consts {
  int path;
  float floor;   // kCopy: what is below becomes 0 (relu: 0, none: -inf)
  float c0, c1;  // kLogistic
  float e0, e1;  // the same times -log2(e), for exp2
};
__device__ inline Consts consts_of(int a) {
  const bool tanh_form = a == kGeluTanh;
  return {a == kGelu ? kNormal : a == kSilu || tanh_form ? kLogistic : kCopy, a == kRelu ? 0.0f : -__builtin_huge_valf(),
          tanh_form ? 1.59576912f : 1.0f, tanh_form ? 0.0713548163f : 0.0f,
          tanh_form ? -2.30220818f : -1.44269504f, tanh_form ? -0.102943240f : 0.0f};
}

// Phi(x) and exp(-x^2 / 2).
__device__ inline float normal_cdf(float x, float* bell) {
  const float a = __builtin_fabsf(x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, a, 1.0f));
  const float e = exp2_fast(-0.72134752f * a * a);
  float r = -0.05023181f;
  r = __builtin_fmaf(r, t, 0.10544527f);
  r = __builtin_fmaf(r, t, 0.0249475f);
  r = __builtin_fmaf(r, t, 0.09445721f);
  r = __builtin_fmaf(r, t, 0.10193547f);
  r = __builtin_fmaf(r, t, 0.11174068f);
  r = __builtin_fmaf(r, t, 0.11170384f);
  const float tail = e * r * t;
  *bell = e;
  return x > 0.0f ? 1.0f - tail : tail;
}

// The square below 10^4, where every s is 0 or 1: silu's constant of 0 times it stays 0, and an x of +inf itself.
__device__ inline float square(float x) { return __builtin_fminf(x * x, 1e4f); }

template <int PATH>
__device__ inline float value(float x, const Consts& c) {
  if constexpr (PATH == kCopy) {
    return x < c.floor ? 0.0f : x;
  } else if constexpr (PATH == kLogistic) {
    return x * __builtin_amdgcn_rcpf(1.0f + exp2_fast(x * __builtin_fmaf(c.e1, square(x), c.e0)));
  } else {
    float bell;
    return x * normal_cdf(x, &bell);
  }
}

// Value and slope. (The backward pass takes as long for these instructions as for its bytes, so they are counted: an
// infinite x has a slope of NaN, which clamping it would avoid. It is that of an infinite sum alone: a finite one is stored
// within its type's range.)
template <int PATH>
__device__ inline float value_and_slope(float x, const Consts& c, float* slope) {
  if constexpr (PATH == kCopy) {
    *slope = c.floor < 0.0f || x > 0.0f ? 1.0f : x != x ? x : 0.0f;
    return x < c.floor ? 0.0f : x;
  } else if constexpr (PATH == kLogistic) {
    const float q = square(x);
    const float p = __builtin_amdgcn_rcpf(1.0f + exp2_fast(x * __builtin_fmaf(c.e1, q, c.e0)));
    const float value = x * p;
    *slope = __builtin_fmaf(value * (1.0f - p), __builtin_fmaf(3.0f * c.c1, q, c.c0), p);
    return value;
  } else {
    float bell;
    const float p = normal_cdf(x, &bell);
    *slope = __builtin_fmaf(0.39894228f * x, bell, p);
    return x * p;
  }
}

// f(path) with the activation's path as a compile-time value.
template <class F>
__device__ inline void with_path(const Consts& c, F f) {
  if (c.path == kCopy) f(std::integral_constant<int, kCopy>{});
  else if (c.path == kLogistic) f(std::integral_constant<int, kLogistic>{});
  else f(std::integral_constant<int, kNormal>{});
}

} // namespace act
} // namespace pgemm
