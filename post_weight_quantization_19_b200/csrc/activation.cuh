// The activation functions of gptq_int8_gated and gptq_activation_int8.
#pragma once

#include <stdint.h>

#include "gptq.h"

namespace gptq {

// In fp32, within 6e-7 of the value: the exponential's two units in the last place, the
// division's two and the roundings.  A NaN stays one.
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == GPTQ_ACT_RELU) return v < 0.f ? 0.f : v;
  if constexpr (ACT == GPTQ_ACT_SILU) return __fdividef(v, 1.f + expf(-v));
  // (not 1 + erf, which cancels for negative v)
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5f * v * erfcf(v * -0.707106781186547524f);
  return v;
}

template <int ACT>
__device__ __forceinline__ double activate64(double v) {
  if constexpr (ACT == GPTQ_ACT_RELU) return v < 0.0 ? 0.0 : v;
  if constexpr (ACT == GPTQ_ACT_SILU) return v / (1.0 + exp(-v));
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5 * v * erfc(v * -0.707106781186547524401);
  return v;
}

}  // namespace gptq
