// gptq_activation_int8: the activation of a feed-forward block in symmetric 8-bit codes with
// one scale per token, what the down projection reads.
//
//   u = act(x) [* up];  scale = max|u| / 127;  code = rint(127 u / max|u|)
//
// ("LLM 量化技术" §1.2, the symmetric quantiser with 8 bits over a token.)  A row's u stay in
// registers in fp32 between the maximum and the codes, so every input is read once and
// every output written once: n d (2 [+ 2 up] + 1 [+ 2 xhat]) bytes.  One CTA per row (rows
// of up to 1024: one warp per row); of rows longer than a CTA's registers hold, the
// rest is read a second time.
//
// Codes are those of the formula in 64 bits.  u is exact in fp32 without an activation and
// with relu (a product of two 16-bit numbers); then what decides a code near a border k +
// 1/2 is the sign of 127 u - (k + 1/2) max|u|, each product taken with its exact
// rounding error (fma), and exact ties go to the even code.  With silu and gelu, u in fp32 is
// off by up to 5e-7 of its value: values that near a border are formed again in 64 bits,
// and so is the row's maximum, from the values within that of the largest.  A row that leaves
// the safe range of fp32, with an infinity or a NaN among them, is done in 64 bits altogether.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "activation_int8.h"
#include "launch_after.h"

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
  static constexpr bool WIDE = false;
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
  static constexpr bool WIDE = true;   // fp32's range
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <int ACT>
constexpr bool EXACT = ACT == GPTQ_ACT_NONE || ACT == GPTQ_ACT_RELU;
// How far a value in fp32 may be off (of it), and 127 u / max|u| with its own roundings.
template <int ACT>
constexpr float VALUE_OFF = 1e-6f;
template <int ACT>
constexpr float QUOTIENT_OFF = EXACT<ACT> ? 5e-7f : 2.f * VALUE_OFF<ACT> + 5e-7f;
// A row is safe with its maximum between these and every |up| at most UP_MOST: values that
// fp32 loses (act below 1e-35, products below 1e-38) then have code 0.
constexpr int STREAM_THREADS = 768;
constexpr size_t STREAM_SMEM = 224 * 1024;
constexpr float LEAST_TOP = 1e-22f, MOST_TOP = 1e36f, UP_MOST = 1e6f;

// The value at an index in 64 bits.  SINGLE: of a row that is safe, and not far below its
// largest.
template <typename T, int ACT, bool SINGLE = true>
__device__ __forceinline__ double value64(const void *x, const void *up, int64_t at) {
  const double f = (double)Half16<T>::one(static_cast<const T *>(x)[at]);
  const double v = SINGLE ? activate64_single<ACT>(f) : activate64<ACT>(f);
  return up ? v * (double)Half16<T>::one(static_cast<const T *>(up)[at]) : v;
}

// `bytes` (a multiple of 16) from 16-byte aligned memory to shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight values of a row in fp32 from their vectors, and `top` raised to their largest
// magnitude, to infinity where the row is not safe (NaN: some value is).
template <typename T, int ACT>
__device__ __forceinline__ void eight_values(const uint4 &x, const uint4 &up, bool gated, float (&u)[8],
                                             float &top) {
  const uint32_t p[4] = {x.x, x.y, x.z, x.w}, q[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Half16<T>::up(p[i]);
    const F2 r = activate_fast<ACT, false>(F2{f.x, f.y});   // (its NaN: a row in 64 bits)
    u[2 * i] = r.x;
    u[2 * i + 1] = r.y;
  }
  if (gated) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Half16<T>::up(q[i]);
      const F2 r = mul2(F2{u[2 * i], u[2 * i + 1]}, F2{f.x, f.y});
      u[2 * i] = r.x;
      u[2 * i + 1] = r.y;
    }
    if constexpr (!EXACT<ACT> && Half16<T>::WIDE) {   // (fp16 does not reach UP_MOST)
      __nv_bfloat162 most = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&q[0]));
#pragma unroll
      for (int i = 1; i < 4; ++i) most = __hmax2(most, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&q[i])));
      if (!(fmaxf(__low2float(most), __high2float(most)) <= UP_MOST)) top = max_or_nan(top, __uint_as_float(0x7F800000u));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_or_nan(top, fabsf(u[i]));
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
    return (float)rint(127.0 * value64<T, ACT>(a.x, a.up, at) / top64);
  }
}

// 1.5 2^23: a sum with it leaves the number rounded to an integer, to even on ties, in the
// low bits.
constexpr float MAGIC = 12582912.f;

// The eight codes of a vector, as MAGIC + code.  `away`: how far from an integer 127 u / max|u|
// may be before a border is near, for every value of this thread.
template <typename T, int ACT>
__device__ __forceinline__ void eight_codes(const ActivationArgs &a, int64_t at, const float (&u)[8], float top,
                                            double top64, float inv, float away, float (&m)[8]) {
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const F2 v{u[i], u[i + 1]}, sum = fma2(v, both(inv), both(MAGIC));
    const F2 c = add2(sum, both(-MAGIC));
    const F2 off = fma2(v, both(-inv), c);
    m[i] = sum.x;
    m[i + 1] = sum.y;
    far = fmaxf(far, fmaxf(fabsf(off.x), fabsf(off.y)));
  }
  if (far >= away) {
    uint32_t near = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = m[i] - MAGIC;
      if (fmaf(fabsf(c), QUOTIENT_OFF<ACT>, fabsf(fmaf(u[i], inv, -c))) >= 0.49999f - QUOTIENT_OFF<ACT>) near |= 1u << i;
    }
#pragma unroll 1
    for (; near; near &= near - 1) {
      const int i = __ffs(near) - 1;
      float ui = u[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) ui = i == k ? u[k] : ui;
      const float code = MAGIC + near_code<T, ACT>(a, at + i, ui, top, top64, ui * inv);
#pragma unroll
      for (int k = 0; k < 8; ++k) m[k] = i == k ? code : m[k];
    }
  }
}

// The low bytes of four MAGIC + code.
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
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
    const double u = fabs(value64<T, ACT, false>(a.x, a.up, row * a.d + k));
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
    if (!lost && top > 0.0) code = (float)rint(127.0 * value64<T, ACT, false>(a.x, a.up, row * a.d + k) / top);
    crow[k] = (int8_t)code;   // |code| <= 127
    if (xh) xh[k] = Half16<T>::put(scale * code);
  }
  return scale;
}

// Where a row's vectors are, and its shared words.
struct RowIn {
  const uint4 *x, *up;
  bool gated;
  uint32_t *words;   // [32]
  double *slot;      // zero
};

// One row: V vectors of eight values per thread in registers, of longer rows (LONG) the
// others formed twice.  `read` is called when no thread reads the row's vectors any more (by
// way of RowIn; values in 64 bits are read from memory).  Returns the scale.
template <typename T, int ACT, int V, bool WARP_ROW, bool LONG, typename Read>
__device__ __forceinline__ float one_row(const ActivationArgs &a, const RowIn &in, int64_t row, int tid, int nt,
                                         int8_t *crow, T *xhrow, double *slots, uint32_t *words, Read read) {
  const int nvec = a.d / 8;
  const uint4 none = make_uint4(0, 0, 0, 0);
  auto values = [&](int k, float (&u)[8], float &top) {
    eight_values<T, ACT>(in.x[k], in.gated ? in.up[k] : none, in.gated, u, top);
  };
  float u[V][8], mine = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int k = min(tid + v * nt, nvec - 1);   // (the last one again: the maximum is the same)
    eight_values<T, ACT>(in.x[k], in.gated ? in.up[k] : none, in.gated, u[v], mine);
  }
  if constexpr (LONG)
    for (int k = tid + V * nt; k < nvec; k += nt) {
      float w[8];
      values(k, w, mine);
    }
  const float top = __uint_as_float(row_max<WARP_ROW>(__float_as_uint(mine) & 0x7FFFFFFFu, in.words));
  if (!(top > LEAST_TOP && top < MOST_TOP)) {
    read();
    return row_in_64_bits<T, ACT, WARP_ROW>(a, row, tid, nt, crow, xhrow, slots, words);
  }
  double top64 = top;
  if constexpr (!EXACT<ACT>) {
    // the largest value in 64 bits: of those that may be it
    const float least = top * (1.f - 3.f * VALUE_OFF<ACT>);
    double m = 0.0;
    if (mine >= least) {
      // (four vectors at a time, a bit for each value that may be it)
#pragma unroll
      for (int v0 = 0; v0 < V; v0 += 4) {
        uint32_t some = 0;
#pragma unroll
        for (int v = v0; v < V && v < v0 + 4; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fabsf(u[v][i]) >= least) some |= 1u << ((v - v0) * 8 + i);
#pragma unroll 1
        for (; some; some &= some - 1) {
          const int b = __ffs(some) - 1;
          m = fmax(m, fabs(value64<T, ACT>(in.x, in.gated ? in.up : nullptr, min(tid + (v0 + b / 8) * nt, nvec - 1) * 8 + b % 8)));
        }
      }
      if constexpr (LONG) {
#pragma unroll 1
        for (int k = tid + V * nt; k < nvec; k += nt) {
          float w[8], wtop = 0.f;
          values(k, w, wtop);
          if (wtop < least) continue;
          uint32_t some = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fabsf(w[i]) >= least) some |= 1u << i;
#pragma unroll 1
          for (; some; some &= some - 1)
            m = fmax(m, fabs(value64<T, ACT>(in.x, in.gated ? in.up : nullptr, k * 8 + __ffs(some) - 1)));
        }
      }
    }
    if constexpr (WARP_ROW) {
      top64 = row_max64<true>(m, nullptr);
    } else {   // few threads have one; non-negative numbers are ordered as their bits
      if (m > 0.0)
        atomicMax(reinterpret_cast<unsigned long long *>(in.slot), (unsigned long long)__double_as_longlong(m));
      __syncthreads();
      top64 = *in.slot;
    }
  }
  if constexpr (!LONG) read();
  const float scale = (float)(top64 * (1.0 / 127.0));   // (good to 2^-52 before it is rounded)
  const float inv = __fdividef(127.f, top), away = 0.49999f - QUOTIENT_OFF<ACT> * fmaf(mine, inv, 1.f);
  auto finish = [&](int k, const float (&w)[8]) {
    float m[8];
    eight_codes<T, ACT>(a, row * a.d + k * 8, w, top, top64, inv, away, m);
    *reinterpret_cast<uint2 *>(crow + (size_t)k * 8) =
        make_uint2(pack_codes(m[0], m[1], m[2], m[3]), pack_codes(m[4], m[5], m[6], m[7]));
    if (xhrow) {
      float c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = scale * (m[i] - MAGIC);
      reinterpret_cast<uint4 *>(xhrow)[k] =
          make_uint4(Half16<T>::down(c[0], c[1]), Half16<T>::down(c[2], c[3]), Half16<T>::down(c[4], c[5]),
                     Half16<T>::down(c[6], c[7]));
    }
  };
  if constexpr (LONG) {
    for (int k = tid + V * nt; k < nvec; k += nt) {
      float w[8], unused = 0.f;
      values(k, w, unused);
      finish(k, w);
    }
    __syncthreads();
    read();
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (tid + v * nt < nvec) finish(tid + v * nt, u[v]);
  return scale;
}

// The scale, and with perm the codes (from shared memory) and xhat in its order.
template <typename T, bool WARP_ROW>
__device__ __forceinline__ void finish_row(const ActivationArgs &a, int64_t row, int tid, int nt, float scale,
                                           const int8_t *crow) {
  if (tid == 0) a.scales[row] = scale;
  if (!a.perm) return;
  if constexpr (WARP_ROW)
    __syncwarp();
  else
    __syncthreads();
  T *xh = static_cast<T *>(a.xhat);
  for (int j = tid; j < a.d; j += nt) {
    const int8_t c = crow[min(max(__ldcg(a.perm + j), 0), a.d - 1)];
    a.codes[row * a.d + j] = c;
    if (xh) xh[row * a.d + j] = Half16<T>::put(scale * (float)c);
  }
}

// A row per CTA or per warp, straight from memory.
template <typename T, int ACT, int V, bool WARP_ROW, bool LONG>
__global__ void __launch_bounds__(WARP_ROW ? 256 : 1024) activation_rows_kernel(const ActivationArgs a) {
  extern __shared__ __align__(16) int8_t row_codes[];   // perm: [rows of the CTA][d]
  __shared__ uint32_t words[3][32];
  __shared__ double slots[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARP_ROW ? lane : (int)threadIdx.x, nt = WARP_ROW ? 32 : (int)blockDim.x;
  const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : (int64_t)blockIdx.x;
  pdl_wait_then_release();
  if (row >= a.n) return;   // whole warps (WARP_ROW) or whole CTAs
  if (!WARP_ROW && tid == 0) slots[0] = 0.0;
  const int nvec = a.d / 8;
  const RowIn in{reinterpret_cast<const uint4 *>(a.x) + row * nvec, reinterpret_cast<const uint4 *>(a.up) + row * nvec,
                 a.up != nullptr, words[0], slots};
  int8_t *crow = a.perm ? row_codes + (WARP_ROW ? (size_t)warp * a.d : 0) : a.codes + row * a.d;
  T *xhrow = a.xhat && !a.perm ? static_cast<T *>(a.xhat) + row * a.d : nullptr;
  const float scale =
      one_row<T, ACT, V, WARP_ROW, LONG>(a, in, row, tid, nt, crow, xhrow, slots, words[1], [] {});
  finish_row<T, WARP_ROW>(a, row, tid, nt, scale, crow);
}

// Many rows: a CTA walks its share of them, and the copy engine brings the next rows to
// shared memory (two at a time) while it works on one.  With loads by the threads
// themselves a CTA alternated between waiting for memory and for its barriers.
template <typename T, int ACT, int V, bool LONG>
__global__ void __launch_bounds__(STREAM_THREADS) activation_stream_kernel(const ActivationArgs a, int *status) {
  extern __shared__ __align__(16) uint8_t stream_smem[];   // two rows of x and up, then perm's codes
  __shared__ uint64_t full[2];
  __shared__ uint32_t words[2][32], words64[2][32];
  __shared__ double slot[2], slots64[32];
  __shared__ int abort;
  const int tid = threadIdx.x, nt = blockDim.x;
  const bool gated = a.up != nullptr;
  const uint32_t half = (uint32_t)a.d * 2, stage = gated ? 2 * half : half;
  auto load = [&](int64_t row, int s) {   // thread 0
    mbar_arrive_expect_tx(&full[s], stage);
    bulk_load(stream_smem + (size_t)s * stage, static_cast<const uint8_t *>(a.x) + row * half, half, &full[s]);
    if (gated)
      bulk_load(stream_smem + (size_t)s * stage + half, static_cast<const uint8_t *>(a.up) + row * half, half,
                &full[s]);
  };
  pdl_wait_then_release();
  if (tid == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    abort = 0;
    fence_mbar_init();
    for (int s = 0; s < 2; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < a.n) load(blockIdx.x + (int64_t)s * gridDim.x, s);
  }
  __syncthreads();
  int i = 0;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, ++i) {
    const int s = i & 1;
    // (words and slots of both parities: a slower thread may still read the last row's)
    if (tid == 0) slot[s] = 0.0;
    if (!*(volatile int *)&abort && !mbar_wait_bounded(&full[s], (uint32_t)(i >> 1) & 1u)) {
      atomicCAS(status, 0, (int)GPTQ_ERR_TIMEOUT);
      *(volatile int *)&abort = 1;   // the rows' results are lost, the barriers are still met
    }
    const uint8_t *src = stream_smem + (size_t)s * stage;
    const RowIn in{reinterpret_cast<const uint4 *>(src), reinterpret_cast<const uint4 *>(src + half), gated, words[s],
                   &slot[s]};
    int8_t *crow = a.perm ? reinterpret_cast<int8_t *>(stream_smem) + 2 * (size_t)stage : a.codes + row * a.d;
    T *xhrow = a.xhat && !a.perm ? static_cast<T *>(a.xhat) + row * a.d : nullptr;
    const int64_t next = row + 2 * (int64_t)gridDim.x;
    const float scale = one_row<T, ACT, V, false, LONG>(a, in, row, tid, nt, crow, xhrow, slots64, words64[0], [&] {
      if (tid == 0 && next < a.n && !*(volatile int *)&abort) load(next, s);
    });
    finish_row<T, false>(a, row, tid, nt, scale, crow);
    // (perm's codes are read by all before the next row's are written: a barrier lies between)
  }
  // copies that nobody waited for: time to land
  if (tid == 0 && *(volatile int *)&abort)
    for (const unsigned long long t0 = global_ns(); global_ns() - t0 < 1000000;) {
    }
}

template <typename T, int ACT, int V, bool WARP_ROW, bool LONG>
int launch_rows(const ActivationArgs &a, int threads, cudaStream_t st) {
  const size_t smem = a.perm ? (size_t)(WARP_ROW ? 8 : 1) * a.d : 0;   // WARP_ROW: d <= 1024
  if constexpr (!WARP_ROW) {
    static std::atomic<bool> attr[64] = {};
    if (a.perm)
      if (const int rc = ensure_smem_attr(activation_rows_kernel<T, ACT, V, WARP_ROW, LONG>, 65536, attr)) return rc;
  }
  const unsigned ctas = (unsigned)(WARP_ROW ? (a.n + 7) / 8 : a.n);
  return launch_after(activation_rows_kernel<T, ACT, V, WARP_ROW, LONG>, ctas, WARP_ROW ? 256 : threads, smem, 1, st, a);
}

template <typename T, int ACT, bool LONG>
int launch_stream(const ActivationArgs &a, int threads, size_t smem, int per_sm, cudaStream_t st) {
  constexpr auto kernel = activation_stream_kernel<T, ACT, 4, LONG>;
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(kernel, STREAM_SMEM, attr)) return rc;
  int *status = device_status_word();
  if (!status) return GPTQ_ERR_CUDA;
  const int64_t fit = (int64_t)num_sms() * per_sm;
  return launch_after(kernel, (unsigned)(a.n < fit ? a.n : fit), threads, smem, 1, st, a, status);
}

template <typename T, int ACT>
int launch_act(const ActivationArgs &a, cudaStream_t st) {
  const int nvec = a.d / 8;
  // Many rows: the copy engine.  For wide rows it pays from one row per SM on, where the
  // others run one or two CTAs to an SM (us, this kernel and the other): 300 x 11008 gated
  // 10.4, 11.1, 1000 x 11008 20.4, 25.8; for narrow ones when its start is spread over
  // many: 2000 x 4096 15.2, 14.2, 4096 x 4096 24.5, 25.3, 1000 x 2048 7.0, 5.5, 10000 x 1024 19.3, 22.3.
  const bool many = a.n > (int64_t)num_sms() * (a.d > 6144 ? 1 : 18);
  if (a.d <= 512 || (a.d <= 1024 && !many)) {
    if (nvec <= 64) return launch_rows<T, ACT, 2, true, false>(a, 0, st);
    return launch_rows<T, ACT, 4, true, false>(a, 0, st);
  }
  auto threads = [&](int v) { return ((nvec + v - 1) / v + 31) / 32 * 32; };
  // two rows in shared memory per CTA, as many CTAs as fit
  const size_t smem = (size_t)a.d * ((a.up ? 8 : 4) + (a.perm ? 1 : 0));
  if (many && smem <= STREAM_SMEM) {
    const int t = threads(4) < STREAM_THREADS ? threads(4) : STREAM_THREADS;
    int per_sm = (int)((224u << 10) / (smem + 2048));
    const int most = 768 / t < 1 ? 1 : 768 / t;
    per_sm = per_sm < 1 ? 1 : per_sm > most ? most : per_sm;
    if (threads(4) <= STREAM_THREADS) return launch_stream<T, ACT, false>(a, t, smem, per_sm, st);
    return launch_stream<T, ACT, true>(a, t, smem, per_sm, st);
  }
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
