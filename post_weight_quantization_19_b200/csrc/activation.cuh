// The activation functions of gptq_int8_gated and gptq_activation_int8.
#pragma once

#include <stdint.h>

#include "gptq.h"

namespace gptq {

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

// In fp32, within 6e-7 of the value (gelu of a negative v: 1e-7 v^2 more, its argument's
// rounding) and, of values that fp32 holds with fewer digits, 3e-43.  A NaN stays one.
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == GPTQ_ACT_RELU) return v < 0.f ? 0.f : v;
  if constexpr (ACT == GPTQ_ACT_SILU) {
    // (of a negative v as v exp(v) / (1 + exp(v)): 1 + exp(-v) passes what has a reciprocal, 2^126,
    // where the value is still 1e-36)
    const float e = expf(-fabsf(v));
    return (v < 0.f ? v * e : v) * reciprocal_approx(1.f + e);
  }
  // (not 1 + erf, which cancels for negative v)
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5f * v * erfcf(v * -0.707106781186547524f);
  return v;
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

// exp(v) within 3e-7 of it, |v| <= 88: 2^t with t = v log2 e rounded, and what v - t ln 2 leaves, a
// few 1e-6 at most, to first order.  (ln 2 as the nearest fp32 number and the rest of it: a fused
// multiply-add rounds once v has cancelled the product.)
__device__ __forceinline__ F2 exp_fast(const F2 &v) {
  const F2 t = mul2(v, both(1.44269504088896341f));
  const F2 rest = fma2(t, both(1.90465430e-9f), fma2(t, both(-0.693147182f), v));
  const F2 e{exp2_approx(t.x), exp2_approx(t.y)};
  return fma2(e, rest, e);
}

// The same functions of two numbers of 16 bits (whose squares are exact) in fewer
// instructions, within 4.3e-7 of the value (of all there are: the tests go through them), values
// below 1e-35 lost.  WHOLE: for arguments of fp32's whole range, infinities among them, of which
// 1e-6 (gelu: and 3.1e-8 v^2, the square's rounding); else silu of a v above 2.3e38 is NaN, and gelu
// of one beyond 1e19.  gelu: erfc(z) exp(z^2) / 2 is t = 1 / (1 + |v| / 4) times a polynomial in
// t, z = |v| / sqrt 2: the one of degree 8 with the least relative error up to |v| = 13.5, by
// reweighted least squares, 7.1e-8 with its coefficients in fp32.
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
    F2 s = mul2(mul2(v, v), both(-0.5f));
    if constexpr (WHOLE) s = F2{fmaxf(s.x, -88.f), fmaxf(s.y, -88.f)};
    const F2 tail = mul2(mul2(t, p), exp_fast(s));
    if constexpr (!WHOLE)   // (4096 x 11008 gated to 8 bits 75.5 us; by a choice as below 78.9)
      return fma2(F2{-fabsf(v.x), -fabsf(v.y)}, tail, F2{fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)});
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

// A polynomial of 2^K coefficients in few dependent steps: neighbours first.
template <int N>
__device__ __forceinline__ double polynomial(const double (&c)[N], double x) {
  double r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = c[i];
#pragma unroll
  for (int n = N; n > 1; n /= 2, x *= x)
#pragma unroll
    for (int i = 0; i < n / 2; ++i) r[i] = fma(r[2 * i + 1], x, r[2 * i]);
  return r[0];
}
// exp(v) to 1e-14 of it, |v| <= 500: 2^k by the exponent's bits, and the Taylor polynomial of
// what is left (at most ln 2 / 2: 0.35^12 / 12! = 7e-15).
__device__ __forceinline__ double exp64(double v) {
  const double k = rint(v * 1.4426950408889634);
  const double x = fma(k, -2.3190468138462996e-17, fma(k, -0.69314718055994529, v));
  const double c[16] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                        1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 0.0, 0.0, 0.0, 0.0};
  const double e = polynomial<16>(c, x);
  return __hiloint2double(__double2hiint(e) + ((int)k << 20), __double2loint(e));
}
// 1 / v to 1e-15 of it, v between 1 and 1e30: fp32's, its error to third order.
__device__ __forceinline__ double reciprocal64(double v) {
  const double r = (double)reciprocal_approx((float)v), e = fma(-v, r, 1.0);
  return fma(r, fma(e, e, e), r);
}

// activate64 for single values of rows that stay inside fp32's range, in fewer dependent
// steps, to 1e-13 of a value of at least 1e-31 (others are not asked for: a u that is not coded as
// 0 is 1e-22 / 254 or more, and up 1e6 at most).  gelu: erfc as in activate_fast, by the
// interpolation in 16 Chebyshev points for |v| up to 14 (2.9e-14), t = 1 / (1 + |v| / 5); exp64
// of a square that is off by 2^-53 of up to 98.  A code's 127 u / max|u| is good to
// 127 (2e-13 + four roundings) < 3e-11.
// (4096 x 11008 gated silu 60.0 us, 500 x 49152 gated gelu 70; with activate64 61.6, 76)
template <int ACT>
__device__ __forceinline__ double activate64_single(double v) {
  if constexpr (ACT == GPTQ_ACT_SILU) return v * reciprocal64(1.0 + exp64(fmin(fmax(-v, -60.0), 80.0)));
  if constexpr (ACT == GPTQ_ACT_GELU) {
    const double w = fmin(fabs(v), 14.0), t = reciprocal64(fma(w, 0.2, 1.0));
    const double c[16] = {0.19703886872887227, 0.14811392565338477, 0.089645541730387301, 0.043455520821440378,
                           0.016455773374037613, 0.0045679510497969589, 0.00076507023977717692, -1.9403485000957232e-06,
                           -3.637628350006139e-05, -5.9469052562377556e-06, 1.2178889043923391e-06, 4.6386159624489665e-07,
                           -4.2375233988423133e-08, -3.0786054594500456e-08, 1.6987087292363867e-09, 1.6516423784196377e-09};
    const double tail = t * polynomial<16>(c, fma(t, 2.714285714285714, -1.714285714285714)) * exp64(-0.5 * w * w);
    return v * (v > 0.0 ? 1.0 - tail : tail);
  }
  return activate64<ACT>(v);
}

}  // namespace gptq
