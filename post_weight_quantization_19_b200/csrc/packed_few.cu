// gptq_packed_linear for few tokens: y = x W^^T + bias, bound by reading the
// packed weights once (r d bits/8 + 8 r G bytes).
//
// A warp multiplies 32 rows of codes (two m16 tiles) with up to 8 or 16 tokens
// on warp-level matrix instructions (mma.sync), whose operands come from
// registers: a code goes from its packed word to an operand in about 1.2
// instructions, with nothing written back to shared or tensor memory on the
// way.  (At 16 tokens these instructions reach about a quarter of the tensor
// rate that tcgen05 has, but the weights' bytes take longer than the products
// up to there.)  Inside a 32-code chunk thread t of a row's four takes codes
// 8t .. 8t+7, so a chunk -- one group -- is two k16 steps (16-bit x) or one k32
// step (8-bit x); the order of k inside a step is free as long as both
// operands agree, and it is chosen so that codes leave their words in pairs.
//
// 16-bit x: the operand is q - z, exact in fp16 and bf16 (code bits placed in
// the mantissa of a power of two M, minus M + z), so only the fp32 sums round;
// each group's sum is scaled by s in fp32.  8-bit x: q and x as integers, sums
// exact, s (sum q x - z sum x) per group; sum x comes from one more product
// with a matrix of ones.
//
// Each warp runs its own ring of cp.async stages of 128 columns (weights, x,
// scales, zeros) and meets the others only at the end: the k range is split
// over the CTA's warps and over a cluster of CTAs, whose partial sums are added
// through distributed shared memory in a fixed order.
#include "packed_linear.h"

namespace gptq {
namespace {

constexpr int FEW_WARPS = 8;
constexpr int KS = 128;        // columns per stage
constexpr int ROWS = 32;       // rows per warp (two m16 tiles)

template <int BITS, int XT, int NT>
struct Few {
  static constexpr bool INT8 = XT == GPTQ_I8;
  // Row strides in shared memory, padded so that the eight rows a warp reads
  // at once fall on different banks.
  static constexpr int WSTRIDE = BITS == 4 ? 80 : BITS == 8 ? 160 : 48;
  static constexpr int XROW = INT8 ? KS : 2 * KS;                 // bytes of a token per stage
  static constexpr int XSTRIDE = INT8 ? 160 : 320;
  static constexpr int WBYTES = ROWS * WSTRIDE;
  static constexpr int SZBYTES = ROWS * 4 * 4 * 2;                // four groups of a stage at most
  static constexpr int STAGES = (BITS == 8 ? 3 : 4) - (NT == 2 && !INT8 ? 1 : 0);
  static int stage_bytes(int tokens) { return WBYTES + SZBYTES + tokens * XSTRIDE; }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

template <int XT>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (XT == GPTQ_F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight codes of thread t's share of chunk c of one row, as they lie in
// the stream (low bits first); 8-bit codes fill both words.
template <int BITS>
__device__ __forceinline__ uint2 row_codes(uint32_t row, int c, int t) {
  if constexpr (BITS == 4) return make_uint2(lds32(row + c * 16 + t * 4), 0);
  if constexpr (BITS == 2) return make_uint2(lds16(row + c * 8 + t * 2), 0);
  if constexpr (BITS == 8) return lds64(row + c * 32 + t * 8);
  if constexpr (BITS == 3) {   // 24 bits from bit 24 t of the chunk's 96
    const int at = (t * 24) >> 5;
    const uint32_t lo = lds32(row + c * 12 + at * 4);
    const uint32_t hi = lds32(row + c * 12 + min(at + 1, 2) * 4);
    return make_uint2(__funnelshift_r(lo, hi, (t * 24) & 31), 0);
  }
}

// M / 2^p + z as a pair of 16-bit numbers, M the power of two whose mantissa
// steps are 1 (1024 in fp16, 128 in bf16): exponent bits, and z in units of the
// last place.
template <int XT>
__device__ __forceinline__ uint32_t base_plus(uint32_t z, int p) {
  const uint32_t v = XT == GPTQ_F16 ? ((25u - p) << 10) + (z << p) : ((134u - p) << 7) + (z << p);
  return v | v << 16;
}

template <int XT>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  if constexpr (XT == GPTQ_F16) {
    const __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a),
                                     *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}

// a 2^-p - b with one rounding (none here: the result is an integer below 2^8)
template <int XT>
__device__ __forceinline__ uint32_t scale_sub2(uint32_t a, int p, uint32_t b) {
  const uint32_t nb = b ^ 0x80008000u;
  const uint32_t k1 = XT == GPTQ_F16 ? (15u - p) << 10 : (127u - p) << 7;
  const uint32_t k = k1 | k1 << 16;
  if constexpr (XT == GPTQ_F16) {
    const __half2 v = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<const __half2 *>(&k),
                              *reinterpret_cast<const __half2 *>(&nb));
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const __nv_bfloat162 v =
        __hfma2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&k),
                *reinterpret_cast<const __nv_bfloat162 *>(&nb));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}

// What q - z needs of a row's zero point.
template <int BITS, int XT>
struct ZeroPoint {
  static constexpr int P = BITS == 4 ? (XT == GPTQ_F16 ? 4 : 0) : BITS == 8 ? 0 : BITS;
  uint32_t z0, zp;   // M + z; M / 2^P + z
  float f;           // 2^23 + z (8-bit codes with bf16)
  __device__ __forceinline__ void set(int z) {
    const uint32_t u = (uint32_t)min(max(z, 0), (1 << BITS) - 1);
    z0 = base_plus<XT>(u, 0);
    if constexpr (P > 0) zp = base_plus<XT>(u, P);
    if constexpr (BITS == 8 && XT == GPTQ_BF16) f = 8388608.f + (float)u;
  }
};

// q - z of eight codes as four pairs: (0,4), (1,5), (2,6), (3,7), or for 8-bit
// codes (0,1), (2,3), (4,5), (6,7).
template <int BITS, int XT>
__device__ __forceinline__ void code_pairs(uint2 w, const ZeroPoint<BITS, XT> &z, uint32_t (&o)[4]) {
  constexpr uint32_t M = XT == GPTQ_F16 ? 0x64006400u : 0x43004300u;
  if constexpr (BITS == 4) {
    if constexpr (XT == GPTQ_F16) {
      const uint32_t h = w.x >> 8;
      o[0] = sub2<XT>((w.x & 0x000F000Fu) | M, z.z0);
      o[1] = scale_sub2<XT>((w.x & 0x00F000F0u) | M, 4, z.zp);
      o[2] = sub2<XT>((h & 0x000F000Fu) | M, z.z0);
      o[3] = scale_sub2<XT>((h & 0x00F000F0u) | M, 4, z.zp);
    } else {   // seven mantissa bits: one nibble at a time
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = sub2<XT>(((w.x >> (4 * i)) & 0x000F000Fu) | M, z.z0);
    }
  } else if constexpr (BITS == 3) {
    // codes 0..3 to the low half, 4..7 to the high half
    const uint32_t v = (w.x & 0x00000FFFu) | ((w.x << 4) & 0x0FFF0000u);
    const uint32_t h = v >> 6;
    o[0] = sub2<XT>((v & 0x00070007u) | M, z.z0);
    o[1] = scale_sub2<XT>((v & 0x00380038u) | M, 3, z.zp);
    o[2] = sub2<XT>((h & 0x00070007u) | M, z.z0);
    o[3] = scale_sub2<XT>((h & 0x00380038u) | M, 3, z.zp);
  } else if constexpr (BITS == 2) {
    const uint32_t v = __byte_perm(w.x, 0, 0x4140);   // byte 0 low, byte 1 high
    const uint32_t h = v >> 4;
    o[0] = sub2<XT>((v & 0x00030003u) | M, z.z0);
    o[1] = scale_sub2<XT>((v & 0x000C000Cu) | M, 2, z.zp);
    o[2] = sub2<XT>((h & 0x00030003u) | M, z.z0);
    o[3] = scale_sub2<XT>((h & 0x000C000Cu) | M, 2, z.zp);
  } else if constexpr (XT == GPTQ_F16) {
    o[0] = sub2<XT>(__byte_perm(w.x, 0x64646464u, 0x4140), z.z0);
    o[1] = sub2<XT>(__byte_perm(w.x, 0x64646464u, 0x4342), z.z0);
    o[2] = sub2<XT>(__byte_perm(w.y, 0x64646464u, 0x4140), z.z0);
    o[3] = sub2<XT>(__byte_perm(w.y, 0x64646464u, 0x4342), z.z0);
  } else {
    // 8 bits do not fit bf16's mantissa beside M: through fp32, whose upper half
    // holds |q - z| <= 255 exactly
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = i < 2 ? w.x : w.y;
      const float a = __uint_as_float(__byte_perm(v, 0x4B000000u, (i & 1) ? 0x7442 : 0x7440)) - z.f;
      const float b = __uint_as_float(__byte_perm(v, 0x4B000000u, (i & 1) ? 0x7443 : 0x7441)) - z.f;
      o[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    }
  }
}

// The eight codes as bytes: {0, 2, 4, 6}, {1, 3, 5, 7} for 4-bit codes, else
// in order.
template <int BITS>
__device__ __forceinline__ uint2 code_bytes(uint2 w) {
  if constexpr (BITS == 8) return w;
  if constexpr (BITS == 4) return make_uint2(w.x & 0x0F0F0F0Fu, (w.x >> 4) & 0x0F0F0F0Fu);
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (BITS == 3) {
      const uint32_t v = i ? w.x >> 12 : w.x;
      const uint32_t u = (v & 0x3Fu) | ((v << 10) & 0x003F0000u);
      o[i] = (u & 0x00070007u) | ((u << 5) & 0x07000700u);
    } else {
      const uint32_t v = i ? w.x >> 8 : w.x;
      const uint32_t u = (v & 0xFu) | ((v << 12) & 0x000F0000u);
      o[i] = (u & 0x00030003u) | ((u << 6) & 0x03000300u);
    }
  }
  return make_uint2(o[0], o[1]);
}

struct FewArgs {
  PackedArgs p;
  int ctas_k;        // CTAs of a cluster, along k
  int tokens;        // staged tokens per warp: min(n, 8 NT)
  int stage_bytes;   // of one stage of one warp
  int aligned;       // rows of codes start on 16-byte boundaries
  int fine;          // groups end inside a stage: four (scale, zero) per row and stage
};

template <int BITS, int XT, int NT>
__global__ void __launch_bounds__(32 * FEW_WARPS) packed_few_kernel(const FewArgs a) {
  using F = Few<BITS, XT, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int crank = blockIdx.x % a.ctas_k;
  const int64_t row0 = (int64_t)(blockIdx.x / a.ctas_k) * ROWS;
  const int64_t tok0 = (int64_t)blockIdx.y * (8 * NT);
  const int ntok = (int)min((int64_t)(8 * NT), a.p.n - tok0);
  const int d = a.p.d;
  // this warp's stages
  const int total = (d + KS - 1) / KS;
  const int parts = a.ctas_k * FEW_WARPS, part_id = crank * FEW_WARPS + warp;
  const int s0 = (int)((int64_t)total * part_id / parts);
  const int s1 = (int)((int64_t)total * (part_id + 1) / parts);

  const uint32_t ring = smem_u32(smem) + warp * F::STAGES * a.stage_bytes;
  const int64_t wpr = (int64_t)(d / 32) * BITS;   // words per row

  auto issue = [&](int s, int slot) {
    const uint32_t base = ring + slot * a.stage_bytes;
    const int k0 = s * KS, cols = min(KS, d - k0);
    const int wbytes = cols * BITS / 8;            // of a row
    const uint32_t *src = a.p.qweight + (int64_t)(k0 / 32) * BITS;
    if (a.aligned) {
#pragma unroll
      for (int i = 0; i < BITS; ++i) {
        const int p = lane + 32 * i, row = p / BITS, col = (p % BITS) * 16;
        const bool in = row0 + row < a.p.r && col < wbytes;
        cp_async16(base + row * F::WSTRIDE + col,
                   reinterpret_cast<const char *>(src + (in ? (row0 + row) * wpr : 0)) + (in ? col : 0),
                   in ? min(16, wbytes - col) : 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * BITS; ++i) {
        const int p = lane + 32 * i, row = p / (4 * BITS), col = (p % (4 * BITS)) * 4;
        const bool in = row0 + row < a.p.r && col < wbytes;
        cp_async4(base + row * F::WSTRIDE + col,
                  reinterpret_cast<const char *>(src + (in ? (row0 + row) * wpr : 0)) + (in ? col : 0),
                  in ? 4 : 0);
      }
    }
    // scales and zeros: lane = row
    {
      const bool in = row0 + lane < a.p.r;
      const int64_t at = in ? (row0 + lane) * a.p.G : 0;
      const uint32_t sz = base + F::WBYTES + lane * 16;
      if (!a.fine) {
        const int gi = a.p.group > 0 ? k0 / a.p.group : 0;
        cp_async4(sz, a.p.scales + at + gi, in ? 4 : 0);
        cp_async4(sz + ROWS * 16, a.p.zeros + at + gi, in ? 4 : 0);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int gi = min((k0 + 32 * c) / a.p.group, a.p.G - 1);
          cp_async4(sz + c * 4, a.p.scales + at + gi, in ? 4 : 0);
          cp_async4(sz + ROWS * 16 + c * 4, a.p.zeros + at + gi, in ? 4 : 0);
        }
      }
    }
    // x
    constexpr int PIECES = F::XROW / 16;
    constexpr int XB = F::INT8 ? 1 : 2;
    const int xbytes = cols * XB;
    for (int p = lane; p < ntok * PIECES; p += 32) {
      const int tok = p / PIECES, col = (p % PIECES) * 16;
      const bool in = col < xbytes;
      cp_async16(base + F::WBYTES + F::SZBYTES + tok * F::XSTRIDE + col,
                 reinterpret_cast<const char *>(a.p.x) + ((tok0 + tok) * d + k0) * XB + (in ? col : 0),
                 in ? 16 : 0);
    }
  };

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;

#pragma unroll
  for (int i = 0; i < F::STAGES - 1; ++i) {
    if (s0 + i < s1) issue(s0 + i, i);
    cp_commit();
  }
  int slot = 0;
  for (int s = s0; s < s1; ++s) {
    cp_wait<F::STAGES - 2>();
    __syncwarp();
    {
      const int nx = s + F::STAGES - 1;
      int ns = slot + F::STAGES - 1;
      if (ns >= F::STAGES) ns -= F::STAGES;
      if (nx < s1) issue(nx, ns);
      cp_commit();
    }
    const uint32_t base = ring + slot * a.stage_bytes;
    const uint32_t xbase = base + F::WBYTES + F::SZBYTES;
    const uint32_t sz = base + F::WBYTES;
    if constexpr (!F::INT8) {
      float part[2][NT][4];
      ZeroPoint<BITS, XT> zp[2][2];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c == 0 || a.fine) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              zp[m][h].set((int)lds32(sz + ROWS * 16 + (m * 16 + h * 8 + g) * 16 + c * 4));
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[m][j][i] = 0.f;
          }
        }
        uint32_t xb[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (j * 8 + g < ntok) v = lds128(xbase + (j * 8 + g) * F::XSTRIDE + c * 64 + t * 16);
          if constexpr (BITS == 8) {
            xb[j][0] = v.x, xb[j][1] = v.y, xb[j][2] = v.z, xb[j][3] = v.w;
          } else {
            xb[j][0] = __byte_perm(v.x, v.z, 0x5410), xb[j][1] = __byte_perm(v.x, v.z, 0x7632);
            xb[j][2] = __byte_perm(v.y, v.w, 0x5410), xb[j][3] = __byte_perm(v.y, v.w, 0x7632);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t lo[4], hi[4];
          code_pairs<BITS, XT>(row_codes<BITS>(base + (m * 16 + g) * F::WSTRIDE, c, t), zp[m][0], lo);
          code_pairs<BITS, XT>(row_codes<BITS>(base + (m * 16 + 8 + g) * F::WSTRIDE, c, t), zp[m][1], hi);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16<XT>(part[m][j], lo[0], hi[0], lo[1], hi[1], xb[j][0], xb[j][1]);
            mma16<XT>(part[m][j], lo[2], hi[2], lo[3], hi[3], xb[j][2], xb[j][3]);
          }
        }
        if (c == 3 || a.fine) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int sc = a.fine ? c * 4 : 0;
            const float f0 = __uint_as_float(lds32(sz + (m * 16 + g) * 16 + sc));
            const float f1 = __uint_as_float(lds32(sz + (m * 16 + 8 + g) * 16 + sc));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[m][j][0] = fmaf(f0, part[m][j][0], acc[m][j][0]);
              acc[m][j][1] = fmaf(f0, part[m][j][1], acc[m][j][1]);
              acc[m][j][2] = fmaf(f1, part[m][j][2], acc[m][j][2]);
              acc[m][j][3] = fmaf(f1, part[m][j][3], acc[m][j][3]);
            }
          }
        }
      }
    } else {
      int part[2][NT][4], xs[NT][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c == 0 || a.fine) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[0][j][i] = part[1][j][i] = xs[j][i] = 0;
        }
        uint32_t xb[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint2 v = make_uint2(0, 0);
          if (j * 8 + g < ntok) v = lds64(xbase + (j * 8 + g) * F::XSTRIDE + c * 32 + t * 8);
          if constexpr (BITS == 4) {
            xb[j][0] = __byte_perm(v.x, v.y, 0x6420), xb[j][1] = __byte_perm(v.x, v.y, 0x7531);
          } else {
            xb[j][0] = v.x, xb[j][1] = v.y;
          }
          mma8(xs[j], 0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u, xb[j][0], xb[j][1]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint2 lo = code_bytes<BITS>(row_codes<BITS>(base + (m * 16 + g) * F::WSTRIDE, c, t));
          const uint2 hi = code_bytes<BITS>(row_codes<BITS>(base + (m * 16 + 8 + g) * F::WSTRIDE, c, t));
#pragma unroll
          for (int j = 0; j < NT; ++j) mma8(part[m][j], lo.x, hi.x, lo.y, hi.y, xb[j][0], xb[j][1]);
        }
        if (c == 3 || a.fine) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int sc = a.fine ? c * 4 : 0;
            const uint32_t r0 = sz + (m * 16 + g) * 16 + sc, r1 = r0 + 8 * 16;
            const float f0 = __uint_as_float(lds32(r0)), f1 = __uint_as_float(lds32(r1));
            const int z0 = min(max((int)lds32(r0 + ROWS * 16), 0), (1 << BITS) - 1);
            const int z1 = min(max((int)lds32(r1 + ROWS * 16), 0), (1 << BITS) - 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[m][j][0] = fmaf(f0, (float)(part[m][j][0] - z0 * xs[j][0]), acc[m][j][0]);
              acc[m][j][1] = fmaf(f0, (float)(part[m][j][1] - z0 * xs[j][1]), acc[m][j][1]);
              acc[m][j][2] = fmaf(f1, (float)(part[m][j][2] - z1 * xs[j][0]), acc[m][j][2]);
              acc[m][j][3] = fmaf(f1, (float)(part[m][j][3] - z1 * xs[j][1]), acc[m][j][3]);
            }
          }
        }
      }
    }
    if (++slot == F::STAGES) slot = 0;
  }
  cp_wait<0>();

  // ---- the warps' sums, then the cluster's, each in a fixed order
  constexpr int COLS = 8 * NT, CELLS = ROWS * COLS;
  __syncthreads();                                  // every ring is drained
  float *red = reinterpret_cast<float *>(smem);     // [FEW_WARPS][COLS][ROWS]
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[warp * CELLS + (j * 8 + t * 2 + (i & 1)) * ROWS + m * 16 + (i >> 1) * 8 + g] = acc[m][j][i];
  __syncthreads();
  const int per = CELLS / a.ctas_k;                 // cells this CTA finishes
  const int first = crank * per;
  if (a.ctas_k > 1) {
    for (int i = threadIdx.x; i < CELLS; i += blockDim.x) {
      float v = red[i];
#pragma unroll
      for (int w = 1; w < FEW_WARPS; ++w) v += red[w * CELLS + i];
      red[i] = v;                                   // cell i is this thread's alone
    }
    __syncwarp();
    cluster_sync();
  }
  for (int i = first + threadIdx.x; i < first + per; i += blockDim.x) {
    float v = 0.f;
    if (a.ctas_k > 1) {
      for (int k = 0; k < a.ctas_k; ++k) {
        float o;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(cluster_addr(red + i, k)));
        v += o;
      }
    } else {
      v = red[i];
#pragma unroll
      for (int w = 1; w < FEW_WARPS; ++w) v += red[w * CELLS + i];
    }
    const int col = i / ROWS;
    const int64_t row = row0 + i % ROWS;
    if (col < ntok && row < a.p.r) {
      if constexpr (F::INT8) v *= a.p.x_scales[tok0 + col];
      if (a.p.bias) v += load_as_float(a.p.bias, a.p.ytype, row);
      store_float(a.p.y, a.p.ytype, (tok0 + col) * a.p.r + row, v);
    }
  }
  if (a.ctas_k > 1) {                               // the partial sums stay until all have read them
    __syncwarp();
    cluster_sync();
  }
}

template <int BITS, int XT, int NT>
int launch_few(const PackedArgs &p, cudaStream_t st) {
  using F = Few<BITS, XT, NT>;
  FewArgs a{};
  a.p = p;
  a.tokens = (int)(p.n < 8 * NT ? p.n : 8 * NT);
  a.stage_bytes = (F::stage_bytes(a.tokens) + 127) / 128 * 128;
  a.aligned = ((int64_t)(p.d / 32) * BITS) % 4 == 0 && reinterpret_cast<uintptr_t>(p.qweight) % 16 == 0;
  a.fine = p.group > 0 && p.group % KS != 0;
  const size_t red = (size_t)FEW_WARPS * ROWS * 8 * NT * 4;
  size_t smem = (size_t)FEW_WARPS * F::STAGES * a.stage_bytes;
  if (smem < red) smem = red;
  constexpr size_t most = (size_t)FEW_WARPS * F::STAGES *
                          ((F::WBYTES + F::SZBYTES + 8 * NT * F::XSTRIDE + 127) / 128 * 128);
  static_assert(most <= 227 * 1024, "ring too large");
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(packed_few_kernel<BITS, XT, NT>, most > red ? most : red, attr))
    return rc;
  const int64_t tiles = (p.r + ROWS - 1) / ROWS;
  const int64_t blocks = (p.n + 8 * NT - 1) / (8 * NT);
  const int stages = (p.d + KS - 1) / KS;
  // k split over a cluster while the tiles leave SMs idle and every warp keeps two stages
  int ck = 1;
  while (ck < 8 && tiles * blocks * ck < 2 * num_sms() && stages >= 2 * FEW_WARPS * ck * 2) ck *= 2;
  a.ctas_k = ck;
  if (tiles * ck > INT32_MAX || blocks > 65535) return GPTQ_ERR_INVALID_ARG;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ck;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ck), (unsigned)blocks);
  cfg.blockDim = dim3(32 * FEW_WARPS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = ck > 1 ? 1 : 0;
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, packed_few_kernel<BITS, XT, NT>, a);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_last_error(__FILE__, __LINE__, "kernel launch", e);
    return GPTQ_ERR_CUDA;
  }
  return GPTQ_OK;
}

template <int BITS>
int launch_few_bits(const PackedArgs &p, cudaStream_t st) {
  const bool two = p.n > 8;
  if (p.xtype == GPTQ_F16)
    return two ? launch_few<BITS, GPTQ_F16, 2>(p, st) : launch_few<BITS, GPTQ_F16, 1>(p, st);
  if (p.xtype == GPTQ_BF16)
    return two ? launch_few<BITS, GPTQ_BF16, 2>(p, st) : launch_few<BITS, GPTQ_BF16, 1>(p, st);
  return two ? launch_few<BITS, GPTQ_I8, 2>(p, st) : launch_few<BITS, GPTQ_I8, 1>(p, st);
}

}  // namespace

int launch_packed_few(const PackedArgs &p, cudaStream_t st) {
  switch (p.bits) {
    case 2: return launch_few_bits<2>(p, st);
    case 3: return launch_few_bits<3>(p, st);
    case 4: return launch_few_bits<4>(p, st);
    default: return launch_few_bits<8>(p, st);
  }
}

}  // namespace gptq
