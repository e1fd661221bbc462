// gptq_rmsnorm_int8: residual addition, root-mean-square norm, and symmetric
// 8-bit codes with one scale per token.
//
// Mathematics.  h = T(x + residual), u = gamma h / sqrt(mean(h^2) + eps), scale
// = max|u| / 127, code = rint(u / scale) -- the symmetric quantiser of "LLM
// 量化技术" §1.2 with 8 bits over a token.  The factor 1 / sqrt(...) cancels in
// u / scale, so code = rint(gamma h * (127 / max|gamma h|)): one pass over the
// row gathers sum h^2 and max|gamma h| together, and the codes do not wait for
// the square root.
//
// A row stays in registers (packed in its 16-bit type) between that pass and
// the writing of the codes, so every input is read once and every output
// written once: n d (2 [+ 2 residual] + 1 [+ 2 h] [+ 2 xhat]) bytes.  One CTA
// per row, one barrier for both sums (rows of up to 2048: one warp per row).
// Measured: 4096 x 4096 bf16 with residual and xhat 33 us = 4.6 TB/s (0.71 of the
// copy rate); one row of 4096 3.0 us, launch and two latencies.
// Codes are those of the formula in 64 bits: gamma h is exact in fp32 (a product of
// two 16-bit numbers), so 127 gamma h / max|gamma h| in fp32 decides every code
// that is not within 2e-5 of a border k + 1/2, and there the sign of 127 gamma h -
// (k + 1/2) max|gamma h| does, each product taken with its exact rounding error
// (fma).  Exact ties are real (half of the row's maximum lies at 63.5) and go to
// the even code.  At 0.5, 1.5 and 2.5, where a step is most of the value, a tie
// follows u / scale as it comes out in 64 bits instead, with scale = max|u| (1 /
// 127), as torch evaluates it on a GPU (a division by 127 or another order of the
// products may end on the other side): about one row in 300 of 4096 columns.
// That part comes last, when the row's registers are free.
// The sum of squares is in 64 bits (a square is exact in fp32) and the scale rounded once:
// with the sum in fp32, 35 % of the scales, and the xhat near a rounding border with
// them, had another last bit (4096 x 4096 31.9 us so, 33.0 in 64 bits).  A row whose
// squares or products leave the safe fp32 range (bf16 values above 1e18 or products
// below 1e-30, infinities, NaN) is done again in 64 bits altogether.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gptq_internal.h"
#include "overlap.h"

namespace gptq {
namespace {

template <typename T>
struct Cvt;
template <>
struct Cvt<__half> {
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ __half one(float a) { return __float2half_rn(a); }
};
template <>
struct Cvt<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ __nv_bfloat16 one(float a) { return __float2bfloat16_rn(a); }
};

struct NormArgs {
  const void *x, *residual, *gamma;
  const int32_t *perm;
  void *h;
  int8_t *codes;
  float *scales;
  void *xhat;
  int64_t n;
  int d;
  double eps, inv_d;
};

// sum of v in 64 bits and maximum of the non-negative m over the row's threads, in every
// thread; a NaN in m survives (its bits compare above every number's).
struct Part {
  double v;
  uint32_t mb;
};
template <bool WARP_ROW>
__device__ __forceinline__ void row_reduce(double &v, float &m, Part *part) {
  uint32_t mb = __float_as_uint(m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  mb = __reduce_max_sync(0xffffffffu, mb);
  if constexpr (!WARP_ROW) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) part[warp] = Part{v, mb};
    __syncthreads();
    const Part p = lane < nw ? part[lane] : Part{0.0, 0u};
    v = p.v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    mb = __reduce_max_sync(0xffffffffu, p.mb);
  }
  m = __uint_as_float(mb);
}

// top / (127 sqrt(mean)), rounded once: in fp32, and then what that is off by, from
// top^2 - (127 scale)^2 mean in 64 bits.
__device__ __forceinline__ float scale_of(float top, double mean) {
  const float s = top / (127.f * sqrtf((float)mean));
  if (!(s < 3e38f)) return s;
  const float p2 = __uint_as_float(254u * 0x800000u - (__float_as_uint(top) & 0x7F800000u));   // top p2 in [1, 2)
  const double t = (double)(top * p2), u = (double)s * (127.0 * p2);
  const float off = (float)(t * t - u * u * mean) / (2.f * (top * p2) * (top * p2));
  return (float)(s + (double)(s * off));
}

// sum, or maximum of non-negative values, over the row's threads in 64 bits
template <bool WARP_ROW>
__device__ double row_reduce64(double v, bool largest, double *part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    v = largest ? fmax(v, w) : v + w;
  }
  if constexpr (!WARP_ROW) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = lane < nw ? part[lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(0xffffffffu, v, o);
      v = largest ? fmax(v, w) : v + w;
    }
  }
  return v;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  // |value| <= 127 by construction up to one rounding of the quotient; the
  // conversion saturates to [-128, 127]
  uint32_t r;
  int ia = __float2int_rn(a), ib = __float2int_rn(b), ic = __float2int_rn(c), id = __float2int_rn(d);
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(r) : "r"(id), "r"(ic));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %0;" : "+r"(r) : "r"(ib), "r"(ia));
  return r;
}

// 127 p against the border nearest to u = 127 p / top: the code, as a float (the
// even one on the border), and whether p lies on one of the first borders exactly.
__device__ __forceinline__ float near_code(float p, float top, float u, bool &tie) {
  const float border = floorf(u) + 0.5f;
  const float a = 127.f * p, ea = fmaf(127.f, p, -a);            // 127 p = a + ea
  const float b = border * top, eb = fmaf(border, top, -b);      // border top = b + eb
  const float over = (a - b) + (ea - eb);                        // a and b are close: a - b is exact
  if (over == 0.f) {
    tie |= fabsf(border) < 3.f;
    return rintf(border);
  }
  return over > 0.f ? border + 0.5f : border - 0.5f;
}

// The row's ties, decided by u / scale formed in 64 bits and written over the
// codes (and xhat), which the row's threads have stored: two elements at a
// time, h from where it was written or from its terms.
template <typename T, bool WARP_ROW>
__device__ __forceinline__ void settle_ties(const NormArgs &a, int64_t row, int tid, int nt, float top,
                                            float inv, float scale, int8_t *crow, T *xh,
                                            double *part) {
  const int words = a.d / 2;
  const uint32_t *hsrc = reinterpret_cast<const uint32_t *>(a.h ? a.h : a.x) + row * words;
  const uint32_t *res =
      a.h || !a.residual ? nullptr : reinterpret_cast<const uint32_t *>(a.residual) + row * words;
  const uint32_t *gam = reinterpret_cast<const uint32_t *>(a.gamma);
  auto load = [&](int k) {
    uint32_t v = hsrc[k];
    if (res) {
      const float2 f = Cvt<T>::up(v), e = Cvt<T>::up(__ldg(res + k));
      v = Cvt<T>::down(f.x + e.x, f.y + e.y);
    }
    return Cvt<T>::up(v);
  };
  double acc = 0.0;
#pragma unroll 4
  for (int k = tid; k < words; k += nt) {
    const float2 h = load(k);
    acc += (double)h.x * h.x + (double)h.y * h.y;
  }
  const double root = sqrt(row_reduce64<WARP_ROW>(acc, false, part) / a.d + a.eps);
  acc = 0.0;
#pragma unroll 1
  for (int k = tid; k < words; k += nt) {
    const float2 h = load(k), g = Cvt<T>::up(__ldg(gam + k));
    if (fabsf(h.x * g.x) == top) acc = fmax(acc, fabs((double)h.x / root * (double)g.x));
    if (fabsf(h.y * g.y) == top) acc = fmax(acc, fabs((double)h.y / root * (double)g.y));
  }
  const double step = row_reduce64<WARP_ROW>(acc, true, part) * (1.0 / 127.0);
#pragma unroll 1
  for (int k = tid; k < words; k += nt) {
    const float2 h = load(k), g = Cvt<T>::up(__ldg(gam + k));
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const float x = i ? h.y : h.x, y = i ? g.y : g.x, u = x * y * inv;
      bool tie = false;
      if (fabsf(u - rintf(u)) > 0.49998f) (void)near_code(x * y, top, u, tie);
      if (tie) {
        const float code = (float)rint((double)x / root * (double)y / step);
        crow[2 * k + i] = (int8_t)code;   // |code| <= 127
        if (xh) xh[2 * k + i] = Cvt<T>::one(scale * code);
      }
    }
  }
}

// A whole row in 64 bits, scale, codes and xhat; returns the scale (NaN for a row with
// a NaN or an infinity).  The row's threads have stored h.  A function of its own, with
// its arguments by value, so that the other rows' code keeps its registers.
template <typename T, bool WARP_ROW>
__device__ __noinline__ float row_in_64_bits(const NormArgs a, int64_t row, int tid, int nt, int8_t *crow,
                                             T *xh, double *part) {
  const int words = a.d / 2;
  const uint32_t *hsrc = reinterpret_cast<const uint32_t *>(a.h ? a.h : a.x) + row * words;
  const uint32_t *res =
      a.h || !a.residual ? nullptr : reinterpret_cast<const uint32_t *>(a.residual) + row * words;
  const uint32_t *gam = reinterpret_cast<const uint32_t *>(a.gamma);
  double h[2], g[2];
  auto load = [&](int k) {
    uint32_t v = hsrc[k];
    if (res) {
      const float2 f = Cvt<T>::up(v), e = Cvt<T>::up(res[k]);
      v = Cvt<T>::down(f.x + e.x, f.y + e.y);
    }
    const float2 f = Cvt<T>::up(v), e = Cvt<T>::up(gam[k]);
    h[0] = f.x, h[1] = f.y, g[0] = e.x, g[1] = e.y;
  };
  double sum = 0.0, top = 0.0;
#pragma unroll 1
  for (int k = tid; k < words; k += nt) {
    load(k);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const double p = fabs(h[i] * g[i]);     // exact
      sum += h[i] * h[i] + (p < 1e300 ? 0.0 : p);   // an infinity or a NaN in gamma: in the sum too
      top = fmax(top, p);
    }
  }
  sum = row_reduce64<WARP_ROW>(sum, false, part);
  top = row_reduce64<WARP_ROW>(top, true, part);
  const bool lost = !(sum < 1e300);
  const double root = sqrt(sum / a.d + a.eps);
  // max|u| as u is formed below: rounding keeps the order, so it is the largest product's
  double most = 0.0;
  if (!lost && top > 0.0) {
#pragma unroll 1
    for (int k = tid; k < words; k += nt) {
      load(k);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (fabs(h[i] * g[i]) == top) most = fmax(most, fabs(h[i] / root * g[i]));
    }
  }
  const double step = row_reduce64<WARP_ROW>(most, true, part) * (1.0 / 127.0);
  const float scale = lost ? __uint_as_float(0x7FC00000u) : top > 0.0 ? (float)step : 1.f;
  const bool live = !lost && step > 0.0;
#pragma unroll 1
  for (int k = tid; k < words; k += nt) {
    load(k);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float code = live ? (float)fmin(fmax(rint(h[i] / root * g[i] / step), -128.0), 127.0) : 0.f;
      crow[2 * k + i] = (int8_t)code;
      if (xh) xh[2 * k + i] = Cvt<T>::one(scale * code);
    }
  }
  return scale;
}

template <typename T, int V, bool WARP_ROW>
// (40 registers let 1536 threads share an SM; the ties' part spills, not the rest)
__global__ void __maxnreg__(WARP_ROW ? 128 : V <= 2 ? 40 : 64) rmsnorm_int8_kernel(const NormArgs a) {
  extern __shared__ __align__(16) int8_t row_codes[];   // perm: [rows of the CTA][d]
  __shared__ Part part[32];
  __shared__ double part64[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARP_ROW ? lane : (int)threadIdx.x;
  const int nt = WARP_ROW ? 32 : (int)blockDim.x;
  const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : (int64_t)blockIdx.x;
  if (row >= a.n) return;   // whole warps (WARP_ROW) or whole CTAs
  const int nvec = a.d / 8;
  const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + row * nvec;
  const uint4 *res = reinterpret_cast<const uint4 *>(a.residual) + row * nvec;
  const uint4 *gam = reinterpret_cast<const uint4 *>(a.gamma);
  uint4 hv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int k = tid + v * nt;
    hv[v] = k < nvec ? x[k] : make_uint4(0, 0, 0, 0);
  }
  if (a.residual) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = tid + v * nt;
      if (k < nvec) {
        const uint4 rv = res[k];
        const uint32_t p[4] = {hv[v].x, hv[v].y, hv[v].z, hv[v].w};
        const uint32_t q[4] = {rv.x, rv.y, rv.z, rv.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Cvt<T>::up(p[i]), g = Cvt<T>::up(q[i]);
          o[i] = Cvt<T>::down(f.x + g.x, f.y + g.y);
        }
        hv[v] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (a.h) {
    uint4 *h = reinterpret_cast<uint4 *>(a.h) + row * nvec;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = tid + v * nt;
      if (k < nvec) h[k] = hv[v];
    }
  }
  double ss = 0.0;
  float top;
  {
    uint32_t mb = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = tid + v * nt;
      if (k < nvec) {
        const uint4 gv = __ldg(gam + k);
        const uint32_t p[4] = {hv[v].x, hv[v].y, hv[v].z, hv[v].w};
        const uint32_t q[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Cvt<T>::up(p[i]);
          const float2 g = Cvt<T>::up(q[i]);
          mb = max(mb, max(__float_as_uint(f.x * g.x) & 0x7FFFFFFFu, __float_as_uint(f.y * g.y) & 0x7FFFFFFFu));
          ss += (double)(f.x * f.x);
          ss += (double)(f.y * f.y);
        }
      }
    }
    top = __uint_as_float(mb);
  }
  row_reduce<WARP_ROW>(ss, top, part);
  int8_t *crow = a.perm ? row_codes + (WARP_ROW ? (size_t)warp * a.d : 0) : a.codes + row * a.d;
  uint4 *xh = a.perm ? nullptr : reinterpret_cast<uint4 *>(a.xhat);
  T *xhrow = xh ? reinterpret_cast<T *>(xh + row * nvec) : nullptr;
  bool zeros = false;   // a row of zeros (and not of products too small for fp32)
  if (top == 0.f) {
    uint32_t bits = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) bits |= hv[v].x | hv[v].y | hv[v].z | hv[v].w;
    bits &= 0x7FFF7FFFu;
    zeros = WARP_ROW ? !__any_sync(0xffffffffu, bits) : !__syncthreads_or(bits);
  }
  float scale;
  if (zeros || (ss < 1e37 && top < 1e37f && top > 1e-30f)) {
    scale = zeros ? 1.f : scale_of(top, ss * a.inv_d + a.eps);
    const float inv = zeros ? 0.f : 127.f / top;
    // ---- the codes, eight of a vector in two words
    uint2 c[V];
    bool tie = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = tid + v * nt;
      c[v] = make_uint2(0, 0);
      if (k < nvec) {
        const uint4 gv = __ldg(gam + k);
        const uint32_t p[4] = {hv[v].x, hv[v].y, hv[v].z, hv[v].w};
        const uint32_t q[4] = {gv.x, gv.y, gv.z, gv.w};
        float u[8], far = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Cvt<T>::up(p[i]), g = Cvt<T>::up(q[i]);
          u[2 * i] = f.x * g.x * inv;
          u[2 * i + 1] = f.y * g.y * inv;
          far = fmaxf(far, fmaxf(fabsf(u[2 * i] - rintf(u[2 * i])), fabsf(u[2 * i + 1] - rintf(u[2 * i + 1]))));
        }
        if (far > 0.49998f) {   // a border is near
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = Cvt<T>::up(p[i / 2]), g = Cvt<T>::up(q[i / 2]);
            if (fabsf(u[i] - rintf(u[i])) > 0.49998f)
              u[i] = near_code((i & 1) ? f.y * g.y : f.x * g.x, top, u[i], tie);
          }
        }
        c[v].x = pack4(u[0], u[1], u[2], u[3]);
        c[v].y = pack4(u[4], u[5], u[6], u[7]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = tid + v * nt;
      if (k < nvec) {
        *reinterpret_cast<uint2 *>(crow + (size_t)k * 8) = c[v];
        if (xh) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = i < 2 ? c[v].x : c[v].y;
            const int s0 = (i & 1) * 16;
            o[i] = Cvt<T>::down(scale * (float)(int8_t)(w >> s0), scale * (float)(int8_t)(w >> (s0 + 8)));
          }
          xh[row * nvec + k] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    if (WARP_ROW ? __any_sync(0xffffffffu, tie) : __syncthreads_or(tie)) {   // the codes are stored
      if constexpr (WARP_ROW) __syncwarp();
      settle_ties<T, WARP_ROW>(a, row, tid, nt, top, inv, scale, crow, xhrow, part64);
    }
  } else {
    if constexpr (WARP_ROW)
      __syncwarp();
    else
      __syncthreads();   // h is stored
    scale = row_in_64_bits<T, WARP_ROW>(a, row, tid, nt, crow, xhrow, part64);
  }
  if (tid == 0) a.scales[row] = scale;
  if (a.perm) {
    if constexpr (WARP_ROW)
      __syncwarp();
    else
      __syncthreads();
    T *xhp = reinterpret_cast<T *>(a.xhat);
    for (int j = tid; j < a.d; j += nt) {
      int from = __ldg(a.perm + j);
      from = from < 0 ? 0 : (from >= a.d ? a.d - 1 : from);
      const int8_t c = crow[from];
      a.codes[row * a.d + j] = c;
      if (xhp) xhp[row * a.d + j] = Cvt<T>::one(scale * (float)c);
    }
  }
}

template <typename T, int V>
int launch_norm(const NormArgs &a, bool warp_row, int threads, cudaStream_t st) {
  if (warp_row) {
    const size_t smem = a.perm ? (size_t)8 * a.d : 0;   // d <= 2048 V / 8
    rmsnorm_int8_kernel<T, V, true>
        <<<(unsigned)((a.n + 7) / 8), 256, smem, st>>>(a);
  } else {
    static std::atomic<bool> attr[64] = {};
    if (a.perm)
      if (const int rc = ensure_smem_attr(rmsnorm_int8_kernel<T, V, false>, 65536, attr)) return rc;
    rmsnorm_int8_kernel<T, V, false>
        <<<(unsigned)a.n, threads, a.perm ? (size_t)a.d : 0, st>>>(a);
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename T>
int launch_norm_t(const NormArgs &a, cudaStream_t st) {
  const int nvec = a.d / 8;
  if (a.d <= 2048) {
    if (nvec <= 32) return launch_norm<T, 1>(a, true, 0, st);
    if (nvec <= 64) return launch_norm<T, 2>(a, true, 0, st);
    if (nvec <= 128) return launch_norm<T, 4>(a, true, 0, st);
    return launch_norm<T, 8>(a, true, 0, st);
  }
  // Vectors per thread: few where the rows are few and a row's latency counts, two
  // (the CTAs of an SM then wait at their barriers at different times) where they
  // are many.  bf16 with residual and xhat, us: 4096 rows of 4096 35.1 with one, 31.8 with
  // two, 34.4 with four; 2048 of 8192: 50.1, 34.2, 37.3; one row of 4096: 2.8, 3.6, 4.8;
  // 1024 rows of 16384: 43.8 with two (1024 threads), 38.6 with four.  (Before the sums
  // were in 64 bits, which cost all of them 3 %.)
  const bool many = a.n > 2 * (int64_t)num_sms();
  auto threads = [&](int v) { return ((nvec + v - 1) / v + 31) / 32 * 32; };
  if (!many && threads(1) <= 1024) return launch_norm<T, 1>(a, false, threads(1), st);
  if (threads(2) <= (many ? 768 : 1024)) return launch_norm<T, 2>(a, false, threads(2), st);
  if (threads(4) <= 1024) return launch_norm<T, 4>(a, false, threads(4), st);
  return launch_norm<T, 8>(a, false, threads(8), st);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_rmsnorm_int8(const void *x, const void *residual, const void *gamma, int dtype,
                                 int64_t n, int64_t d, double eps, const int32_t *perm, void *h,
                                 int8_t *codes, float *scales, void *xhat, gptq_stream_t stream) {
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (n < 0 || n > (int64_t)INT32_MAX) return GPTQ_ERR_INVALID_ARG;
  if (d <= 0 || d % 32 != 0 || d > 65536) return GPTQ_ERR_INVALID_ARG;
  if (!(eps >= 1e-30) || !(eps <= 1e30)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!x || !gamma || !codes || !scales) return GPTQ_ERR_INVALID_ARG;
  for (const void *p : {x, residual, gamma, (const void *)h, (const void *)codes, (const void *)xhat})
    if (reinterpret_cast<uintptr_t>(p) % 16) return GPTQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(scales) % 4 || reinterpret_cast<uintptr_t>(perm) % 4)
    return GPTQ_ERR_INVALID_ARG;
  // a row's outputs may not be another row's inputs, nor each other
  const size_t row16 = (size_t)n * d * 2;
  const Span in[] = {{x, row16}, {residual, row16}, {gamma, (size_t)d * 2}, {perm, (size_t)d * 4}};
  const Span out[] = {{h, row16}, {codes, (size_t)n * d}, {scales, (size_t)n * 4}, {xhat, row16}};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlap(out[i], out[j])) return GPTQ_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j < 2 && h == in[j].p)) return GPTQ_ERR_INVALID_ARG;
  }
  const NormArgs a{x, residual, gamma, perm, h, codes, scales, xhat, n, (int)d, eps, 1.0 / (double)d};
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == GPTQ_F16 ? launch_norm_t<__half>(a, st) : launch_norm_t<__nv_bfloat16>(a, st);
}
