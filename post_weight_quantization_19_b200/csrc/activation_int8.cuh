// gptq_activation_int8: the activation of a feed-forward block in symmetric 8-bit codes with
// one scale per token, what the down projection reads.
//
//   u = act(x) [* up];  scale = max|u| / 127;  code = rint(127 u / max|u|)
//
// ("LLM 量化技术" §1.2, the symmetric quantiser with 8 bits over a token.)  A row's u stay in
// registers in fp32 between the maximum and the codes, so every input is read once and
// every output written once: n d (2 [+ 2 up] + 1 [+ 2 xhat]) bytes.  One CTA per row (rows
// of up to 2048: one warp per row); of rows longer than a CTA's registers hold, the
// rest is read a second time.
//
// Codes are those of the formula in 64 bits.  u is exact in fp32 without an activation and
// with relu (a product of two 16-bit numbers); then what decides a code near a border k +
// 1/2 is the sign of 127 u - (k + 1/2) max|u|, each product taken with its exact
// rounding error (fma), and exact ties go to the even code.  With silu and gelu, u in fp32 is
// off by up to 6e-7 (gelu: 2e-5, at arguments around -13) of its value: values that
// near a border are formed again in 64 bits, and so is the row's maximum, from the
// values within that of the largest.  A row that leaves the safe range of fp32, with an
// infinity or a NaN among them, is done in 64 bits altogether.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "activation_int8.h"

namespace gptq {
namespace {

template <typename T>
struct Half16;
template <>
struct Half16<__half> {
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <int ACT>
constexpr bool EXACT = ACT == GPTQ_ACT_NONE || ACT == GPTQ_ACT_RELU;
// How far a value in fp32 may be off, and twice that of 127 u / max|u|.
template <int ACT>
constexpr float VALUE_OFF = ACT == GPTQ_ACT_GELU ? 2e-5f : 6e-7f;
template <int ACT>
constexpr float QUOTIENT_OFF = 2.f * VALUE_OFF<ACT> + 3e-7f;
// A row is safe with its maximum between these and every |up| at most UP_MOST: values that
// fp32 loses (act below 3e-37, products below 1e-38) then have code 0.
constexpr float LEAST_TOP = 1e-24f, MOST_TOP = 1e36f, UP_MOST = 1e6f;

// Value i of a row in 64 bits.
template <typename T, int ACT>
__device__ __forceinline__ double value64(const ActivationArgs &a, int64_t at) {
  const double v = activate64<ACT>((double)Half16<T>::one(static_cast<const T *>(a.x)[at]));
  return a.up ? v * (double)Half16<T>::one(static_cast<const T *>(a.up)[at]) : v;
}

// Eight values of a row in fp32 from their vectors; the largest magnitude's bits are returned,
// an infinity's where the row is not safe.
template <typename T, int ACT>
__device__ __forceinline__ uint32_t eight_values(const uint4 &x, const uint4 &up, bool gated, float (&u)[8]) {
  const uint32_t p[4] = {x.x, x.y, x.z, x.w}, q[4] = {up.x, up.y, up.z, up.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Half16<T>::up(p[i]);
    u[2 * i] = activate<ACT>(f.x);
    u[2 * i + 1] = activate<ACT>(f.y);
  }
  if (gated) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Half16<T>::up(q[i]);
      u[2 * i] *= f.x;
      u[2 * i + 1] *= f.y;
      most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    if (!EXACT<ACT> && !(most <= UP_MOST)) top = 0x7F800000u;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(u[i]) & 0x7FFFFFFFu);
  return top;
}

// The code of u near a border, as a float.
template <typename T, int ACT>
__device__ __forceinline__ float near_code(const ActivationArgs &a, int64_t at, float u, float top, double top64,
                                           float q) {
  if constexpr (EXACT<ACT>) {
    const float border = floorf(q) + 0.5f;
    const float m = 127.f * u, em = fmaf(127.f, u, -m);         // 127 u = m + em
    const float b = border * top, eb = fmaf(border, top, -b);   // border top = b + eb
    const float over = (m - b) + (em - eb);                     // m and b are close: m - b is exact
    return over == 0.f ? rintf(border) : over > 0.f ? border + 0.5f : border - 0.5f;
  } else {
    return (float)rint(127.0 * value64<T, ACT>(a, at) / top64);
  }
}

// The eight codes of a vector, as floats.
template <typename T, int ACT>
__device__ __forceinline__ void eight_codes(const ActivationArgs &a, int64_t at, const float (&u)[8], float top,
                                            double top64, float inv, float (&c)[8]) {
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = u[i] * inv;
    c[i] = rintf(q);
    // (over 1/2 - the quotient's error: a border is near)
    far = fmaxf(far, fmaf(fabsf(q), EXACT<ACT> ? 4e-7f : QUOTIENT_OFF<ACT>, fabsf(q - c[i])));
  }
  if (far >= 0.5f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float ui = u[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) ui = i == k ? u[k] : ui;
      const float q = ui * inv, n = rintf(q);
      if (fmaf(fabsf(q), EXACT<ACT> ? 4e-7f : QUOTIENT_OFF<ACT>, fabsf(q - n)) < 0.5f) continue;
      const float code = near_code<T, ACT>(a, at + i, ui, top, top64, q);
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = i == k ? code : c[k];
    }
  }
}

__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  uint32_t r;
  const int ia = __float2int_rn(a), ib = __float2int_rn(b), ic = __float2int_rn(c), id = __float2int_rn(d);
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(r) : "r"(id), "r"(ic));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %0;" : "+r"(r) : "r"(ib), "r"(ia));
  return r;
}

// Largest of a value's bits over the row's threads, in every thread.  `slot`: one word
// per warp of shared memory, used once between barriers.
template <bool WARP_ROW>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *slot) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (!WARP_ROW) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    v = __reduce_max_sync(0xffffffffu, lane < nw ? slot[lane] : 0u);
  }
  return v;
}
// The same of non-negative numbers in 64 bits (no NaN).
template <bool WARP_ROW>
__device__ __forceinline__ double row_max64(double v, double *slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (!WARP_ROW) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    v = lane < nw ? slot[lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

// A whole row in 64 bits; returns the scale.  Arguments by value, so that the other rows'
// code keeps its registers.
template <typename T, int ACT, bool WARP_ROW>
__device__ __noinline__ float row_in_64_bits(const ActivationArgs a, int64_t row, int tid, int nt, int8_t *crow,
                                             T *xh, double *slot, uint32_t *words) {
  double top = 0.0;
  bool lost = false, any = false;
  // a row of zeros, as padding leaves them: no value in 64 bits is needed
#pragma unroll 4
  for (int k = tid; k < a.d; k += nt) {
    const float f = Half16<T>::one(static_cast<const T *>(a.x)[row * a.d + k]);
    const float g = a.up ? Half16<T>::one(static_cast<const T *>(a.up)[row * a.d + k]) : 1.f;
    any |= !((f == 0.f || (ACT == GPTQ_ACT_RELU && f < 0.f)) && fabsf(g) < 1e38f) && !(g == 0.f && fabsf(f) < 1e38f);
  }
  if (row_max<WARP_ROW>(any ? 1u : 0u, words) == 0) {
#pragma unroll 4
    for (int k = tid; k < a.d; k += nt) {
      crow[k] = 0;
      if (xh) xh[k] = Half16<T>::put(0.f);
    }
    return 1.f;
  }
#pragma unroll 1
  for (int k = tid; k < a.d; k += nt) {
    const double u = fabs(value64<T, ACT>(a, row * a.d + k));
    if (u <= 1.7e308)
      top = fmax(top, u);
    else
      lost = true;
  }
  top = row_max64<WARP_ROW>(top, slot);
  lost = row_max<WARP_ROW>(lost ? 1u : 0u, words + 32) != 0;
  const float scale = lost ? __uint_as_float(0x7FC00000u) : top > 0.0 ? (float)(top / 127.0) : 1.f;
#pragma unroll 1
  for (int k = tid; k < a.d; k += nt) {
    float code = 0.f;
    if (!lost && top > 0.0) code = (float)rint(127.0 * value64<T, ACT>(a, row * a.d + k) / top);
    crow[k] = (int8_t)code;   // |code| <= 127
    if (xh) xh[k] = Half16<T>::put(scale * code);
  }
  return scale;
}

// V vectors of eight values per thread in registers.  LONG: the row's other vectors are
// formed twice.
template <typename T, int ACT, int V, bool WARP_ROW, bool LONG>
__global__ void __launch_bounds__(WARP_ROW ? 256 : 1024) activation_int8_kernel(const ActivationArgs a) {
  extern __shared__ __align__(16) int8_t row_codes[];   // perm: [rows of the CTA][d]
  __shared__ uint32_t words[3][32];
  __shared__ double slot[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARP_ROW ? lane : (int)threadIdx.x, nt = WARP_ROW ? 32 : (int)blockDim.x;
  const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : (int64_t)blockIdx.x;
  if (row >= a.n) return;   // whole warps (WARP_ROW) or whole CTAs
  const int nvec = a.d / 8;
  const bool gated = a.up != nullptr;
  const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + row * nvec;
  const uint4 *up = reinterpret_cast<const uint4 *>(a.up) + row * nvec;
  const uint4 none = make_uint4(0, 0, 0, 0);
  float u[V][8];
  uint32_t mb = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int k = tid + v * nt;
    const uint4 xv = k < nvec ? __ldg(x + k) : none, uv = gated && k < nvec ? __ldg(up + k) : none;
    mb = max(mb, eight_values<T, ACT>(xv, uv, gated, u[v]));
  }
  if constexpr (LONG)
    for (int k = tid + V * nt; k < nvec; k += nt) {
      float w[8];
      mb = max(mb, eight_values<T, ACT>(__ldg(x + k), gated ? __ldg(up + k) : none, gated, w));
    }
  const float top = __uint_as_float(row_max<WARP_ROW>(mb, words[0]));
  int8_t *crow = a.perm ? row_codes + (WARP_ROW ? (size_t)warp * a.d : 0) : a.codes + row * a.d;
  T *xhrow = a.xhat && !a.perm ? static_cast<T *>(a.xhat) + row * a.d : nullptr;
  float scale;
  if (top > LEAST_TOP && top < MOST_TOP) {
    double top64 = top;
    if constexpr (!EXACT<ACT>) {
      // the largest value in 64 bits: of those that may be it
      const float least = top * (1.f - 3.f * VALUE_OFF<ACT>);
      double m = 0.0;
      if (__uint_as_float(mb) >= least) {
#pragma unroll 1
        for (int k = tid; k < nvec; k += nt) {
          float w[8];
          (void)eight_values<T, ACT>(__ldg(x + k), gated ? __ldg(up + k) : none, gated, w);
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            float wi = w[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) wi = i == j ? w[j] : wi;
            if (fabsf(wi) >= least) m = fmax(m, fabs(value64<T, ACT>(a, row * a.d + k * 8 + i)));
          }
        }
      }
      top64 = row_max64<WARP_ROW>(m, slot);
    }
    scale = (float)(top64 / 127.0);
    const float inv = 127.f / top;
    auto finish = [&](int k, const float (&w)[8]) {
      float c[8];
      eight_codes<T, ACT>(a, row * a.d + k * 8, w, top, top64, inv, c);
      *reinterpret_cast<uint2 *>(crow + (size_t)k * 8) =
          make_uint2(pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7]));
      if (xhrow)
        reinterpret_cast<uint4 *>(xhrow)[k] =
            make_uint4(Half16<T>::down(scale * c[0], scale * c[1]), Half16<T>::down(scale * c[2], scale * c[3]),
                       Half16<T>::down(scale * c[4], scale * c[5]), Half16<T>::down(scale * c[6], scale * c[7]));
    };
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (tid + v * nt < nvec) finish(tid + v * nt, u[v]);
    if constexpr (LONG)
      for (int k = tid + V * nt; k < nvec; k += nt) {
        float w[8];
        (void)eight_values<T, ACT>(__ldg(x + k), gated ? __ldg(up + k) : none, gated, w);
        finish(k, w);
      }
  } else {
    scale = row_in_64_bits<T, ACT, WARP_ROW>(a, row, tid, nt, crow, xhrow, slot, words[1]);
  }
  if (tid == 0) a.scales[row] = scale;
  if (a.perm) {
    if constexpr (WARP_ROW)
      __syncwarp();
    else
      __syncthreads();
    T *xhp = static_cast<T *>(a.xhat);
    for (int j = tid; j < a.d; j += nt) {
      const int8_t c = crow[min(max(__ldg(a.perm + j), 0), a.d - 1)];
      a.codes[row * a.d + j] = c;
      if (xhp) xhp[row * a.d + j] = Half16<T>::put(scale * (float)c);
    }
  }
}

template <typename T, int ACT, int V, bool WARP_ROW, bool LONG>
int launch_rows(const ActivationArgs &a, int threads, cudaStream_t st) {
  const size_t smem = a.perm ? (size_t)(WARP_ROW ? 8 : 1) * a.d : 0;   // WARP_ROW: d <= 2048
  if constexpr (!WARP_ROW) {
    static std::atomic<bool> attr[64] = {};
    if (a.perm)
      if (const int rc = ensure_smem_attr(activation_int8_kernel<T, ACT, V, WARP_ROW, LONG>, 65536, attr)) return rc;
  }
  const unsigned ctas = (unsigned)(WARP_ROW ? (a.n + 7) / 8 : a.n);
  activation_int8_kernel<T, ACT, V, WARP_ROW, LONG><<<ctas, WARP_ROW ? 256 : threads, smem, st>>>(a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename T, int ACT>
int launch_act(const ActivationArgs &a, cudaStream_t st) {
  const int nvec = a.d / 8;
  if (a.d <= 2048) {
    if (nvec <= 64) return launch_rows<T, ACT, 2, true, false>(a, 0, st);
    return launch_rows<T, ACT, 8, true, false>(a, 0, st);
  }
  auto threads = [&](int v) { return ((nvec + v - 1) / v + 31) / 32 * 32; };
  if (threads(2) <= 1024) return launch_rows<T, ACT, 2, false, false>(a, threads(2), st);
  return launch_rows<T, ACT, 2, false, true>(a, 1024, st);
}

template <typename T>
int launch_activation(const ActivationArgs &a, cudaStream_t st) {
  switch (a.activation) {
    case GPTQ_ACT_NONE: return launch_act<T, GPTQ_ACT_NONE>(a, st);
    case GPTQ_ACT_RELU: return launch_act<T, GPTQ_ACT_RELU>(a, st);
    case GPTQ_ACT_SILU: return launch_act<T, GPTQ_ACT_SILU>(a, st);
    default: return launch_act<T, GPTQ_ACT_GELU>(a, st);
  }
}

}  // namespace
}  // namespace gptq
