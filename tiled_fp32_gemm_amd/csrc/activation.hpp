// activation.hpp -- the activations of include/sgemm_linear.h and their
// derivatives, in FP32.
//
// exp(x) is formed as 2^(x log2 e) with the part of x log2 e that its FP32
// rounding drops added back to first order (exp_accurate): without it the
// relative error of exp grows with |x|.
//
// The normal distribution function.  For a >= 0,
//      Phi(-a) = exp(-a^2 / 2) g(a),   g(a) = exp(a^2 / 2) erfc(a / sqrt 2) / 2,
// and g falls smoothly from 1/2 like 1 / a, so it is a low-degree polynomial in
// t = 1 / (1 + 0.29 a).  The coefficients are a weighted least-squares fit of
// degree 8 over 0 <= a <= 14, iterated towards equal errors: 1.2e-9 absolute
// (times the exponential) before rounding.  Phi(a) = 1 - Phi(-a).  Both tails
// keep their relative accuracy, which 1 + erf would cancel away.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/sgemm_linear.h"

namespace sg {

__device__ __forceinline__ float exp_accurate(float x) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;
  const float hi = x * kLog2e;
  // Past +-104 the result is inf or 0; the clamp keeps the low part of an
  // infinite x from becoming NaN.
  const float c = fminf(fmaxf(x, -104.0f), 104.0f);
  const float lo = fmaf(c, kLog2e, -(c * kLog2e)) + c * kLog2eLow;
  return __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.693147182f, 1.0f);
}

// Phi(z) and exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  const float a = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.29f, a, 1.0f));
  float g = 0.0369796716f;
  g = fmaf(g, t, -0.180613316f);
  g = fmaf(g, t, 0.279229191f);
  g = fmaf(g, t, -0.1186813609f);
  g = fmaf(g, t, 0.1622325786f);
  g = fmaf(g, t, 0.0870671229f);
  g = fmaf(g, t, 0.1182330764f);
  g = fmaf(g, t, 0.1155530375f);
  bell = exp_accurate(-0.5f * z * z);
  const float tail = g * t * bell;
  return z < 0.0f ? tail : 1.0f - tail;
}

// 1 / (1 + exp(-x)).
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_accurate(-x));
}

// The same and 1 - it, both without cancellation.
__device__ __forceinline__ float sigmoid_both(float x, float& rest) {
  const float q = exp_accurate(-fabsf(x));
  const float big = __builtin_amdgcn_rcpf(1.0f + q), small = q * big;
  rest = x >= 0.0f ? small : big;
  return x >= 0.0f ? big : small;
}

constexpr float kTwoSqrt2OverPi = 1.59576912f;    // 2 sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.398942280f;       // 1 / sqrt(2 pi)
constexpr float kTanhCubic = 0.044715f;

// z, but finite, for a factor of a tail that vanishes: inf * 0 becomes 0.
// (NaN becomes finite as well; the other factor keeps it.)
__device__ __forceinline__ float finite(float z) {
  return fminf(fmaxf(z, -1.0e18f), 1.0e18f);
}
// The same for the lower tail only.
__device__ __forceinline__ float above(float z) { return fmaxf(z, -1.0e18f); }

template <int act>
__device__ __forceinline__ float activate(float z) {
  if (act == SGEMM_ACT_RELU) return z <= 0.0f ? 0.0f : z;   // NaN stays NaN
  if (act == SGEMM_ACT_GELU) {
    float bell;
    return above(z) * normal_cdf(z, bell);
  }
  if (act == SGEMM_ACT_GELU_TANH)
    return above(z) * sigmoid(kTwoSqrt2OverPi * z * fmaf(kTanhCubic * z, z, 1.0f));
  if (act == SGEMM_ACT_SILU) return above(z) * sigmoid(z);
  return z;
}

template <int act>
__device__ __forceinline__ float activation_slope(float z) {
  if (act == SGEMM_ACT_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);
  if (act == SGEMM_ACT_GELU) {
    float bell;
    const float cdf = normal_cdf(z, bell);
    return fmaf(finite(z) * kInvSqrt2Pi, bell, cdf);
  }
  if (act == SGEMM_ACT_GELU_TANH) {
    float rest;
    const float s = sigmoid_both(kTwoSqrt2OverPi * z * fmaf(kTanhCubic * z, z, 1.0f), rest);
    // s (1 - s) is 0 in FP32 well before |z| = 30.
    const float c = fminf(fmaxf(z, -30.0f), 30.0f);
    const float du = kTwoSqrt2OverPi * fmaf(3.0f * kTanhCubic * c, c, 1.0f);
    return fmaf(c * du, s * rest, s);
  }
  if (act == SGEMM_ACT_SILU) {
    float rest;
    const float s = sigmoid_both(z, rest);
    return s * fmaf(finite(z), rest, 1.0f);
  }
  return 1.0f;
}

// f(integral_constant<int, act>): a loop for each activation, rather than a
// choice for each element.
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
  switch (act) {
    case SGEMM_ACT_RELU: f(std::integral_constant<int, SGEMM_ACT_RELU>()); break;
    case SGEMM_ACT_GELU: f(std::integral_constant<int, SGEMM_ACT_GELU>()); break;
    case SGEMM_ACT_GELU_TANH: f(std::integral_constant<int, SGEMM_ACT_GELU_TANH>()); break;
    case SGEMM_ACT_SILU: f(std::integral_constant<int, SGEMM_ACT_SILU>()); break;
    default: f(std::integral_constant<int, SGEMM_ACT_NONE>());
  }
}

}  // namespace sg
