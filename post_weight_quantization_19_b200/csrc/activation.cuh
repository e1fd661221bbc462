// The activation functions of gptq_int8_gated and gptq_activation_int8.
#pragma once

#include <stdint.h>

#include "gptq.h"

namespace gptq {

// In fp32, within 6e-7 of the value (gelu of a negative v: 1e-7 v^2 more, its argument's
// rounding).  A NaN stays one.
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == GPTQ_ACT_RELU) return v < 0.f ? 0.f : v;
  if constexpr (ACT == GPTQ_ACT_SILU) return __fdividef(v, 1.f + expf(-v));
  // (not 1 + erf, which cancels for negative v)
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5f * v * erfcf(v * -0.707106781186547524f);
  return v;
}

__device__ __forceinline__ float exp2_approx(float v) {   // within 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal_approx(float v) {   // within 2^-23; 0 above 2^126
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// exp(v) within 4e-7 of it, v <= 88: 2^t with t = v log2 e rounded, and what t is off by, a few
// 1e-6 at most, to first order (ln 2 in two parts).
__device__ __forceinline__ float exp_fast(float v) {
  const float t = v * 1.44269504088896341f;
  const float rest = fmaf(t, -1.42860677e-6f, fmaf(t, -0.693145751953125f, v));
  const float e = exp2_approx(t);
  return fmaf(e, rest, e);
}

// The same functions of a number of 16 bits (its square is exact) in fewer instructions, within
// 8e-7 of the value, values below 1e-35 lost.  gelu: erfc(z) = t exp(-z^2 + P(t)), t = 1 /
// (1 + z / 2), the Chebyshev fit of Numerical Recipes (Press et al., "Error
// function"), good to 1.2e-7 of the value for every z >= 0.
template <int ACT>
__device__ __forceinline__ float activate_fast(float v) {
  if constexpr (ACT == GPTQ_ACT_SILU) return v * reciprocal_approx(1.f + exp_fast(fminf(-v, 88.f)));
  if constexpr (ACT == GPTQ_ACT_GELU) {
    const float t = reciprocal_approx(fmaf(fabsf(v), 0.353553390593273762f, 1.f));
    float p = fmaf(t, 0.17087277f, -0.82215223f);
    p = fmaf(t, p, 1.48851587f);
    p = fmaf(t, p, -1.13520398f);
    p = fmaf(t, p, 0.27886807f);
    p = fmaf(t, p, -0.18628806f);
    p = fmaf(t, p, 0.09678418f);
    p = fmaf(t, p, 0.37409196f);
    p = fmaf(t, p, 1.00002368f);
    p = fmaf(t, p, -1.26551223f);
    // (beyond 13.2 the half tail is below 1e-38)
    const float tail = 0.5f * t * exp_fast(p) * exp_fast(fmaxf(v * v * -0.5f, -88.f));
    return v * (v > 0.f ? 1.f - tail : tail);
  }
  return activate<ACT>(v);
}

template <int ACT>
__device__ __forceinline__ double activate64(double v) {
  if constexpr (ACT == GPTQ_ACT_RELU) return v < 0.0 ? 0.0 : v;
  if constexpr (ACT == GPTQ_ACT_SILU) return v / (1.0 + exp(-v));
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5 * v * erfc(v * -0.707106781186547524401);
  return v;
}

}  // namespace gptq
