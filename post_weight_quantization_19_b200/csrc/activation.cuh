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
// Two fp32 numbers that one instruction works on.
struct F2 {
  float x, y;
};
__device__ __forceinline__ uint64_t bits(const F2 &a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ F2 numbers(uint64_t v) {
  F2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 both(float v) { return F2{v, v}; }
__device__ __forceinline__ F2 fma2(const F2 &a, const F2 &b, const F2 &c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return numbers(r);
}
__device__ __forceinline__ F2 mul2(const F2 &a, const F2 &b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return numbers(r);
}
__device__ __forceinline__ F2 add2(const F2 &a, const F2 &b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return numbers(r);
}

// exp(v) within 4e-7 of it, |v| <= 88: 2^t with t = v log2 e rounded, and what t is off by, a
// few 1e-6 at most, to first order (ln 2 in two parts).
__device__ __forceinline__ F2 exp_fast(const F2 &v) {
  const F2 t = mul2(v, both(1.44269504088896341f));
  const F2 rest = fma2(t, both(-1.42860677e-6f), fma2(t, both(-0.693145751953125f), v));
  const F2 e{exp2_approx(t.x), exp2_approx(t.y)};
  return fma2(e, rest, e);
}

// The same functions of two numbers of 16 bits (whose squares are exact) in fewer
// instructions, within 4.3e-7 of the value (of all there are), values below 1e-35 lost.
// WHOLE: for arguments of fp32's whole range, infinities among them; else silu of a v above
// 2.3e38 is NaN.  gelu: erfc(z) exp(z^2)
// / 2 is t = 1 / (1 + |v| / 4) times a polynomial in t, z = |v| / sqrt 2: the one of degree
// 8 with the least relative error (5e-8) up to |v| = 13.5, by reweighted least squares.
template <int ACT, bool WHOLE>
__device__ __forceinline__ F2 activate_fast(const F2 &v) {
  if constexpr (ACT == GPTQ_ACT_SILU) {
    F2 m{fminf(-v.x, 88.f), fminf(-v.y, 88.f)};
    if constexpr (WHOLE) m = F2{fmaxf(m.x, -88.f), fmaxf(m.y, -88.f)};
    const F2 e = add2(exp_fast(m), both(1.f));
    return mul2(v, F2{reciprocal_approx(e.x), reciprocal_approx(e.y)});
  }
  if constexpr (ACT == GPTQ_ACT_GELU) {
    const F2 z = fma2(F2{fabsf(v.x), fabsf(v.y)}, both(0.25f), both(1.f));
    const F2 t{reciprocal_approx(z.x), reciprocal_approx(z.y)};
    F2 p = fma2(t, both(0.0262750126f), both(-0.155535161f));
    p = fma2(t, p, both(0.301862329f));
    p = fma2(t, p, both(-0.212497279f));
    p = fma2(t, p, both(0.206518233f));
    p = fma2(t, p, both(0.0308376569f));
    p = fma2(t, p, both(0.104300849f));
    p = fma2(t, p, both(0.0984358788f));
    p = fma2(t, p, both(0.0998024642f));
    // (beyond 13.2 the half tail is below 1e-38)
    const F2 s = mul2(mul2(v, v), both(-0.5f));
    const F2 tail = mul2(mul2(t, p), exp_fast(F2{fmaxf(s.x, -88.f), fmaxf(s.y, -88.f)}));
    const F2 rest = fma2(tail, both(-1.f), both(1.f));
    return mul2(v, F2{v.x > 0.f ? rest.x : tail.x, v.y > 0.f ? rest.y : tail.y});
  }
  return F2{activate<ACT>(v.x), activate<ACT>(v.y)};
}

template <int ACT>
__device__ __forceinline__ double activate64(double v) {
  if constexpr (ACT == GPTQ_ACT_RELU) return v < 0.0 ? 0.0 : v;
  if constexpr (ACT == GPTQ_ACT_SILU) return v / (1.0 + exp(-v));
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5 * v * erfc(v * -0.707106781186547524401);
  return v;
}

}  // namespace gptq
