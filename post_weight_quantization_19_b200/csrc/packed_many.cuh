// gptq_packed_linear for many tokens: y = x W^^T + bias on the 5th-generation
// tensor cores, the weights dequantised on their way into tensor memory.
//
// Up to 192 tokens, and a few hundred of small layers: one CTA per tile of 128 rows
// of W and N <= 192 tokens.  More: a pair of CTAs per tile of 256 rows and N <= 192
// tokens, or twice as many in two accumulators that share the weights' conversion.  The weights are the MMA's A
// operand, in tensor memory: TMA brings blocks of 128 rows x 256 columns of codes to
// shared memory (rows that are not multiples of 16 bytes: cp.async; threads that each
// copied their own row's 32 bytes ran at half the speed), and thread i of a converter
// warpgroup, which owns row i, turns 64 columns of it into 16-bit weights and writes
// them to its TMEM lane (tcgen05.st).  x is the B operand: tiles of 64 features x N tokens that TMA
// places in 128-byte-swizzled shared memory.  So shared memory carries x and the
// codes, not the weights, and a code costs about 2.5 instructions once per tile.
// In a pair each CTA loads half of the tokens' x and the MMAs (cta_group::2) read
// both halves: without pairs every CTA loaded all of its x from L2, 64 KB per 1024
// clocks of MMAs for 256 tokens, and L2's bandwidth was the bound (4096 tokens x 4096
// x 11008: 287 us when pairs made it 241; 512 tokens x 8192 x 8192: 65.5 and 57.6).
//
//   w = T16(s (q - z)):  q - z is exact in 16 bits (code bits in the mantissa of
//   a power of two M, minus M + z); s is split in two 16-bit parts, so w =
//   fma(q - z, s_hi, (q - z) s_lo) is s (q - z) rounded once (up to the second
//   part's own rounding, 2^-10 of half a step).  This rounding is
//   gptq_dequant_fp16's; fp32 weights would need three times the tensor work.
//   With fp16, s is multiplied by a power of two per row (that brings the largest weight
//   to fp16's upper range) and the row's sums divided by it again, so scales outside
//   fp16's range lose nothing, nor those far below the row's largest.
//
// Warp 0 loads x, warp 1 issues the MMAs, warps 2-3 load codes, scales and zeros;
// warps 4-19 are four converter warpgroups, one for each 64 columns of a block;
// warps 20-23 drain the accumulators, one while the other fills (23 ns a token; with
// two accumulators that share weights nothing fills meanwhile.  The converter warps'
// help there cost their own loop registers, and more time than it saved).  Single CTAs
// with fewer tiles than SMs split the k range over a cluster, whose CTAs add their
// sums through distributed shared memory in a fixed order.
//
// Measured (4 bits, groups of 128): 4096 tokens x 4096 x 11008, bf16, 247 to 252 us in a
// burst = 1480 TFLOP/s (0.89 of the measured burst rate), 292 us under the power cap;
// 1000 tokens of 8-bit x, 11008 x 4096, 82 us (129 tiles over 74 pairs of SMs are two
// rounds); 64 tokens x 4096 x 4096, 13.3 us, bound by start, fill and the cluster's sums.
//
// fp32 results (FP32): a weight s (q - z) enters as an fp32 number, the sum of two fp16 or
// three bf16 parts that the MMAs take one after the other with the same x, and a sum
// leaves the tensor core every 256 features: its additions truncate, and over a whole
// row that was 5e-5 to 1e-4 too little where all products have one sign (65536 features,
// 40 and 300 tokens of fp16; 1e-5 with exact weights), now 2e-6.  The drain warps add those
// sums up in tensor memory, behind two accumulators of 128 tokens.  4096 tokens x 4096 x
// 11008 take 1041 us with fp16 and 1573 with bf16, bound by conversion (1600 clocks a
// part and step); sums of 512 features take 4 % less, adding to y itself half as long again.
// For 16-bit results a sum stays for all of a CTA's features: 1.5e-5 to 3e-5 too little at
// 11008, 1e-4 at 65536, where half a step of fp16 is 2.4e-4 to 4.9e-4.
#pragma once

#include <mutex>

#include "packed_linear.h"

namespace gptq {
namespace {

constexpr int PM = 128;                 // rows of W per tile (UMMA M)
constexpr int PN = 192;                 // most tokens per tile (UMMA N)
constexpr int PK = 64;                  // features per box of x (one 128-byte row)
constexpr int SK = 2 * PK;              // features per step: two boxes, eight MMAs
constexpr int ASTAGES = 2;              // TMEM stages of A: 64 columns each
constexpr int MAXB = 6;                 // shared-memory stages of x at most
constexpr uint32_t TM_A = 2 * PN;       // TMEM column of the first A stage
constexpr int WGS = 4;                  // converter warpgroups
constexpr int MANY_THREADS = 32 * (4 + 4 * WGS + 4);
constexpr size_t MANY_SMEM = 217 * 1024;   // x and codes, after alignment

constexpr int BLK = 2;                  // steps per block of codes; a warpgroup takes half a step
constexpr int BCOLS = BLK * SK;         // its columns
constexpr int LOADERS = 64;
// FP32: most tokens per tile, and the place of a tile's sums in tensor memory, behind two
// accumulators that take a block of codes each
constexpr int PN32 = 128;
constexpr uint32_t TM_SUM = 2 * PN32;
static_assert(TM_SUM + PN32 <= TM_A, "sums and A stages overlap");
static_assert(ASTAGES == BLK && WGS == 2 * BLK, "step j of a block uses A stage j");

// A block of codes in shared memory, as TMA lays it down: boxes of 128 rows x up
// to 128 bytes, 16-byte chunks exchanged inside 128 bytes (TMA's 128- and 64-byte
// swizzles) so that the rows that a quarter-warp reads at once fall on different
// banks; 3-bit rows of 96 bytes have no swizzle.  Then scales [sub][row] and
// zeros [sub][row] of its `subs` parts of equal group.
template <int BITS>
struct CodeBlock {
  static constexpr int ROW = BCOLS * BITS / 8;      // bytes of a row
  static constexpr int BOX = ROW < 128 ? ROW : 128; // of it in a box
  static constexpr int CODES = PM * ROW;
  // place of byte `col` (16-byte chunks move as one) of a row
  static __device__ __forceinline__ uint32_t place(int row, int col) {
    if constexpr (BITS == 3) return row * ROW + col;
    const int c = (col % BOX) >> 4, x = BOX == 128 ? row & 7 : (row >> 1) & 3;
    return (col / BOX) * (PM * BOX) + row * BOX + ((c ^ x) << 4) + (col & 15);
  }
  static constexpr int DEPTH = BITS == 8 ? 2 : 3;
  static __host__ __device__ constexpr int bytes(int subs) { return CODES + PM * 8 * subs; }
};

struct ManyArgs {
  PackedArgs p;
  int N;              // tokens per accumulator, a multiple of 16
  int halves;         // accumulators per tile: 1, or 2 that share the converted weights
  int nM, nN;         // tiles
  int ctas_k;         // CTAs of a cluster, along k
  int bstages;
  int aligned;        // 16-byte loads of the codes
  uint32_t gdiv;      // ceil(2^31 / (group / 32)), 0 for one group
  int subs;           // parts of a block that lie in one group each: 1, 2, 4 or 8
  int *status;
};

struct ManyShared {
  uint64_t full_b[MAXB], empty_b[MAXB];
  uint64_t full_a[ASTAGES], empty_a[ASTAGES];
  uint64_t full_c[3], empty_c[3];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  uint32_t exponent[2][PM];   // fp16: safe_exponent of a tile's rows
  alignas(16) uint4 stage[4][64];   // results on their way out, per warp
  alignas(16) float scale[4][PN];   // and the scales of x's tokens
};

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands, fp32 accumulate.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The same over a pair of CTAs: each CTA's 128 rows of A and D in its own tensor
// memory, half of B's tokens in the shared memory of each.
__device__ __forceinline__ void umma_f16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void many_timeout(int *status, ManyShared &sh) {
  atomicCAS(status, 0, (int)GPTQ_ERR_TIMEOUT);
  *(volatile int *)&sh.abort = 1;
}

// Pairs of 16-bit numbers in a register.
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
  static constexpr uint32_t M = 0x64006400u;   // 1024: mantissa steps of 1
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    const __half2 v = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 v = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b),
                              *reinterpret_cast<__half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint32_t both(float s) {
    const __half2 v = __half2half2(__float2half_rn(s));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ float low(uint32_t v) {
    return __low2float(*reinterpret_cast<const __half2 *>(&v));
  }
};
template <>
struct Pair<__nv_bfloat16> {
  static constexpr uint32_t M = 0x43004300u;   // 128
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v =
        __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v =
        __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    const __nv_bfloat162 v =
        __hfma2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b),
                *reinterpret_cast<__nv_bfloat162 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint32_t both(float s) {
    const __nv_bfloat162 v = __bfloat162bfloat162(__float2bfloat16_rn(s));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ float low(uint32_t v) { return __uint_as_float(v << 16); }
};

// A group's scale and zero point, ready for code pairs.
template <int BITS, typename T>
struct Group {
  uint32_t mz, hi, lo;   // M + z; s = hi + lo
  float s, z;            // 8-bit codes in bf16: through fp32
  __device__ __forceinline__ void set(float scale, int zero) {
    const uint32_t u = (uint32_t)min(max(zero, 0), (1 << BITS) - 1);
    if constexpr (BITS == 8 && sizeof(T) == 2 && Pair<T>::M == 0x43004300u) {
      s = scale;
      z = 8388608.f + (float)u;
    } else {
      mz = Pair<T>::M + (u | u << 16);
      hi = Pair<T>::both(scale);
      const float rest = scale - Pair<T>::low(hi);
      lo = Pair<T>::both(rest == rest ? rest : 0.f);   // inf - inf: hi carries it
    }
  }
  __device__ __forceinline__ uint32_t weight(uint32_t magic_plus_q) const {
    const uint32_t v = Pair<T>::sub(magic_plus_q, mz);
    return Pair<T>::fma(v, hi, Pair<T>::mul(v, lo));
  }
};

// 32 codes of one row and group as 16 pairs of weights, in column order.
// `magic`: M in a register that the compiler does not see through, so that mask and
// M take one instruction (which holds one constant).
template <int BITS, typename T>
__device__ __forceinline__ void chunk_weights(const uint32_t *w, const Group<BITS, T> &g,
                                              uint32_t magic, uint32_t (&o)[16]) {
  constexpr uint32_t M = Pair<T>::M;
  if constexpr (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = w[i], h = v >> 4;   // byte k: codes 2k (low nibble of v), 2k + 1 (of h)
      o[4 * i + 0] = g.weight((__byte_perm(v, h, 0x0400) & 0x000F000Fu) | magic);
      o[4 * i + 1] = g.weight((__byte_perm(v, h, 0x0501) & 0x000F000Fu) | magic);
      o[4 * i + 2] = g.weight((__byte_perm(v, h, 0x0602) & 0x000F000Fu) | magic);
      o[4 * i + 3] = g.weight((__byte_perm(v, h, 0x0703) & 0x000F000Fu) | magic);
    }
  } else if constexpr (BITS == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w[i], h = v >> 2;
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // byte k: codes 4k .. 4k + 3
        const uint32_t b = __byte_perm(v, h, 0x0400 + 0x0101 * k);
        o[8 * i + 2 * k] = g.weight((b & 0x00030003u) | magic);
        o[8 * i + 2 * k + 1] = g.weight(((b >> 4) & 0x00030003u) | magic);
      }
    }
  } else if constexpr (BITS == 3) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {   // six bits from stream bit 6 i
      const int pos = 6 * i, wi = pos >> 5, off = pos & 31;
      const uint32_t v = off + 6 > 32 ? __funnelshift_r(w[wi], w[wi + 1], off) : w[wi] >> off;
      o[i] = g.weight((v & 7u) | ((v << 13) & 0x00070000u) | magic);
    }
  } else if constexpr (M == 0x64006400u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[2 * i] = g.weight(__byte_perm(w[i], 0x64646464u, 0x4140));
      o[2 * i + 1] = g.weight(__byte_perm(w[i], 0x64646464u, 0x4342));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t v = w[i >> 1];
      const float a = __uint_as_float(__byte_perm(v, 0x4B000000u, (i & 1) ? 0x7442 : 0x7440)) - g.z;
      const float b = __uint_as_float(__byte_perm(v, 0x4B000000u, (i & 1) ? 0x7443 : 0x7441)) - g.z;
      const __nv_bfloat162 p = __floats2bfloat162_rn(a * g.s, b * g.s);
      o[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
  }
}

// Part `P` of the weights of 32 codes of one row and group in fp32, s (q - z), as 16
// pairs in column order: the number rounded to fp16 and then the rest; in bf16 its
// upper, middle and lower 8 bits.  What the parts before it hold is formed again
// rather than kept: registers are short.
template <int BITS, typename T, int P>
__device__ __forceinline__ void chunk_part(const uint32_t *w, float s, float z, uint32_t (&o)[16]) {
  auto code = [&](int j) {   // 2^23 + q
    const int pos = j * BITS, wi = pos >> 5, off = pos & 31;
    const uint32_t v = off + BITS > 32 ? __funnelshift_r(w[wi], w[wi + 1], off) : w[wi] >> off;
    return __uint_as_float((v & ((1u << BITS) - 1u)) | 0x4B000000u);
  };
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a = (code(2 * i) - z) * s, b = (code(2 * i + 1) - z) * s;
    if constexpr (Pair<T>::M == 0x64006400u) {
      __half2 h = __floats2half2_rn(a, b);
      if constexpr (P == 1) h = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
      o[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
        b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
      }
      o[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    }
  }
}

// Group of the 32-column chunk c of a row.
__device__ __forceinline__ int group_of(const ManyArgs &a, int c) {
  return (int)(((uint64_t)(uint32_t)c * a.gdiv) >> 31);
}

// fp16: a row's scales are multiplied by 2^(LIFT + 127 - e), with e the exponent bits of
// the largest one (from the bits of its magnitude), and its sums by the reciprocal:
// the largest weights, below 2^(LIFT + 1 + BITS) = 2^15, fill fp16's range, so that groups
// with scales of up to 2^(LIFT + 14) less than the row's largest are still normal numbers.
template <int BITS>
constexpr uint32_t LIFT = 14 - BITS;
template <int BITS>
__device__ __forceinline__ uint32_t safe_exponent(uint32_t top) {
  return min(max(top >> 23, LIFT<BITS> + 1u), 253u);
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ uint32_t pair_of(const __half *, float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pair_of(const __nv_bfloat16 *, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// One accumulator of a warp's 32 rows, `count` tokens from t0 with scales `scale`, to
// y.  A lane is a row; 16-bit results go as pairs of tokens through 1 KB of shared
// memory, 16 tokens of 32 rows at a time, and out 16 bytes (8 rows of a token) per
// lane, where y's rows allow it: storing them as they lie cost 100 clocks a token.
// True if a result is not a number's (fp32 results only).
template <typename Y>
__device__ __forceinline__ bool write_tile(uint32_t base, int count, float f, float bias,
                                           const float *scale, int64_t t0, int64_t row,
                                           const PackedArgs &p, uint4 *stage, int lane) {
  Y *y = static_cast<Y *>(p.y) + t0 * p.r + row;
  const bool live = row < p.r;
  bool wide = false, lost = false;
  if constexpr (sizeof(Y) == 2)
    wide = p.r % 8 == 0 && row - lane + 32 <= p.r && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
  Y *yw = y - lane + (lane & 3) * 8 + (int64_t)(lane >> 2) * 2 * p.r;   // this lane's 8 rows of two tokens
  for (int c0 = 0; c0 < count; c0 += 16) {
    float v[16];
    tmem_ld_32x32b_x16(base + c0, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], f * scale[c0 + i], bias);
    if (wide) {
      if constexpr (sizeof(Y) == 2) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<uint32_t *>(stage)[i * 32 + lane] = pair_of(y, v[2 * i], v[2 * i + 1]);
        __syncwarp();
        const uint4 a = stage[2 * lane], b = stage[2 * lane + 1];
        Y *at = yw + (int64_t)c0 * p.r;
        const int tok = c0 + (lane >> 2) * 2;
        if (tok < count)
          *reinterpret_cast<uint4 *>(at) =
              make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                         __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
        if (tok + 1 < count)
          *reinterpret_cast<uint4 *>(at + p.r) =
              make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                         __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (live && c0 + i < count) {
          put(y + (int64_t)(c0 + i) * p.r, v[i]);
          if constexpr (sizeof(Y) == 4) lost |= !(fabsf(v[i]) <= 3.402823466e38f);
        }
    }
  }
  return lost;
}

// FP32: a warp's 32 rows of an accumulator's N sums added to those in `total`, or with
// `first` put there.
__device__ __forceinline__ void add_sums(uint32_t total, uint32_t base, int N, bool first) {
  for (int c0 = 0; c0 < N; c0 += 16) {
    float v[16], w[16];
    tmem_ld_32x32b_x16(base + c0, v);
    if (!first) tmem_ld_32x32b_x16(total + c0, w);
    tmem_wait_ld();
    uint32_t o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(first ? v[i] : v[i] + w[i]);
    tmem_st_x16(total + c0, o);
  }
  tmem_wait_st();
}

// FP32: a result again, from its definition, if it is not a number's (an infinity times
// two parts of a weight with different signs is none).  By value, as settle_lost.
template <int BITS>
__device__ __noinline__ void settle_result(const PackedArgs p, int64_t tok, int64_t row) {
  float *y = static_cast<float *>(p.y) + tok * p.r + row;
  if (fabsf(*y) <= 3.402823466e38f) return;
  if (p.x_scales && !(fabsf(p.x_scales[tok]) <= 3.402823466e38f)) return;   // the token's scale is none
  float v = sum_in_64_bits<BITS>(p, tok, row);
  if (p.x_scales) v *= p.x_scales[tok];
  *y = p.bias ? v + static_cast<const float *>(p.bias)[row] : v;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

template <int BITS, typename T, bool PAIR, bool FP32>
__global__ void __launch_bounds__(MANY_THREADS, 1)
    packed_many_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmW, const ManyArgs a) {
  constexpr bool HALF = Pair<T>::M == 0x64006400u;
  constexpr int PARTS = !FP32 ? 1 : HALF ? 2 : 3;   // of a weight
  static_assert(!(PAIR && FP32), "fp32 results come from single CTAs");
  using C = CodeBlock<BITS>;
  extern __shared__ uint8_t dyn_smem[];
  __shared__ ManyShared sh;
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // PAIR: two CTAs, `rank` 0 (which issues the MMAs) and 1, with a row tile each
  // and half of the tokens' x.  Otherwise ctas_k CTAs share a tile along k.
  const int N = a.N, box_bytes = (PAIR ? N / 2 : N) * PK * 2, bstage_bytes = 2 * box_bytes;
  const int rank = PAIR ? (int)cluster_rank() : 0, sharing = PAIR ? 2 : a.ctas_k;
  const int crank = PAIR ? 0 : blockIdx.x % a.ctas_k;
  const int ctas = gridDim.x / sharing, cta = blockIdx.x / sharing;
  const int nMt = PAIR ? (a.nM + 1) / 2 : a.nM;
  const int tiles = nMt * a.nN;
  // first row of this CTA in tile t (past the last row for an odd pair's second CTA)
  auto first_row = [&](int t) { return (int64_t)(PAIR ? t % nMt * 2 + rank : t % nMt) * PM; };
  const int total = (a.p.d + SK - 1) / SK, blocks = (total + BLK - 1) / BLK;
  const int kb0 = (int)((int64_t)blocks * crank / a.ctas_k);          // this CTA's blocks
  const int kb1 = (int)((int64_t)blocks * (crank + 1) / a.ctas_k);
  const int ks0 = kb0 * BLK, ks1 = min(kb1 * BLK, total);             // and steps

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAXB; ++s) {
      mbar_init(&sh.full_b[s], 1);
      mbar_init(&sh.empty_b[s], 1);
    }
    for (int s = 0; s < ASTAGES; ++s) {
      mbar_init(&sh.full_a[s], PAIR ? 16 : 8);
      mbar_init(&sh.empty_a[s], 1);
    }
    for (int c = 0; c < C::DEPTH; ++c) {
      mbar_init(&sh.full_c[c], LOADERS + 1);
      mbar_init(&sh.empty_c[c], 4 * WGS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], PAIR ? 8 : 4);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmX);
    if (a.aligned) prefetch_tmap(&tmW);
  }
  __syncwarp();
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&sh.tmem_base, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sh.tmem_base, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();   // both CTAs' barriers before either signals the other
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  bool settle = false;   // FP32: a result of this thread's is not a number's

  if (warp == 0) {
    // ---------------------------------------------------------------- x by TMA
    if (lane == 0) {
      if (a.p.follows) asm volatile("griddepcontrol.wait;" ::: "memory");   // x; the codes are there
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      bool ok = true;
      for (int t = cta; t < tiles && ok; t += ctas) {
        const int n0 = (t / nMt) * (N * a.halves) + rank * (N / 2);
        for (int q = ks0 * a.halves; q < ks1 * a.halves; ++q) {
          const int ks = a.halves == 2 ? q >> 1 : q, h = a.halves == 2 ? q & 1 : 0;
          if (*(volatile int *)&sh.abort) {
            ok = false;
            break;
          }
          if (!mbar_wait_bounded(&sh.empty_b[stage], phase ^ 1)) {
            many_timeout(a.status, sh);
            ok = false;
            break;
          }
          if (rank == 0) {
            mbar_arrive_expect_tx(&sh.full_b[stage], PAIR ? 2 * bstage_bytes : bstage_bytes);
            issued |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          }
          // feature offsets: multiples of 64 16-bit values = 128 bytes (past d: zeros)
          uint8_t *dst = smem + (size_t)stage * bstage_bytes;
          if constexpr (PAIR) {   // counted on the issuing CTA's barrier
            const uint32_t bar = cluster_addr(&sh.full_b[stage], 0);
            tma_load_2d_pair(dst, &tmX, ks * SK, n0 + h * N, bar);
            tma_load_2d_pair(dst + box_bytes, &tmX, ks * SK + PK, n0 + h * N, bar);
          } else {
            tma_load_2d(dst, &tmX, ks * SK, n0 + h * N, &sh.full_b[stage]);
            tma_load_2d(dst + box_bytes, &tmX, ks * SK + PK, n0 + h * N, &sh.full_b[stage]);
          }
          if (++stage == a.bstages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      for (int s = 0; s < MAXB; ++s)
        if (issued & (1u << s)) (void)mbar_wait_bounded(&sh.full_b[s], (issued_par >> s) & 1u);
      // a second CTA whose loads the other may not have waited for: time to land
      if (PAIR && rank == 1 && !ok)
        for (const unsigned long long t0 = global_ns(); global_ns() - t0 < 1000000;) {
        }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- the MMAs
    // The whole warp walks the loop, so that what the MMAs take (tensor-memory
    // addresses, descriptors) stays in uniform registers, and one elected thread
    // issues them; with a lone thread in the loop each MMA cost 60 clocks to
    // issue, as long as 120 tokens take to multiply.  Descriptors advance by
    // constants (16-byte units); a step is eight MMAs per accumulator.
    const uint32_t fmt = HALF ? 0u : 1u;
    const uint32_t idesc = instr_desc(fmt, fmt, 0, 0, PAIR ? 2 * PM : PM, N);
    const uint64_t first = smem_desc(smem_u32(smem), 16, 1024, 2);
    const uint32_t box = (uint32_t)box_bytes >> 4;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const bool two = a.halves == 2;
    uint64_t bdesc = first;
    int bstage = 0;
    uint32_t bphase = 0, aphase = 0, abuf = 0, cphase = 0;   // aphase, cphase: a bit per stage
    bool ok = true;
    // the MMAs of one step and accumulator
    auto issue = [&](uint32_t buf, int j, bool fresh, bool last, bool frees_a) {
      if (fresh) ok = mbar_wait_bounded(&sh.acc_empty[buf], ((cphase >> buf) & 1u) ^ 1u);
      ok = ok && mbar_wait_bounded(&sh.full_b[bstage], bphase);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t dt = tm + buf * PN, ad = tm + TM_A + j * (SK / 2);
        auto mma = [&](uint32_t at, uint64_t desc, uint32_t accumulate) {
          if constexpr (PAIR)
            umma_f16_pair_ts(dt, at, desc, idesc, accumulate);
          else
            umma_f16_ts(dt, at, desc, idesc, accumulate);
        };
        auto commit = [&](uint64_t *bar) {
          if constexpr (PAIR)
            umma_commit_both(bar);
          else
            umma_commit(bar);
        };
        mma(ad, bdesc, fresh ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < 4; ++kk) mma(ad + kk * 8, bdesc + kk * 2, 1u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma(ad + 32 + kk * 8, bdesc + box + kk * 2, 1u);
        commit(&sh.empty_b[bstage]);
        if (frees_a) commit(&sh.empty_a[j]);
        if (last) commit(&sh.acc_full[buf]);
      }
      __syncwarp();
      if (last) cphase ^= 1u << buf;
      bdesc += 2 * box;
      if (++bstage == a.bstages) {
        bstage = 0;
        bphase ^= 1;
        bdesc = first;
      }
    };
    if constexpr (FP32) {
      // The two steps of a block in turn, part after part, so that one A stage is
      // written while the other is multiplied; the block's x stays for all parts.
      auto stage_of = [&](int j, uint32_t &ph) {
        const int s = bstage + j;
        ph = s < a.bstages ? bphase : bphase ^ 1u;
        return s < a.bstages ? s : s - a.bstages;
      };
      for (int t = cta; t < tiles && ok; t += ctas) {
        for (int kb = kb0; kb < kb1 && ok; ++kb) {
          const int count = min(BLK, ks1 - kb * BLK);
          ok = mbar_wait_bounded(&sh.acc_empty[abuf], ((cphase >> abuf) & 1u) ^ 1u);
          for (int q = 0; q < PARTS * count && ok; ++q) {
            const int j = q % count, part = q / count;
            uint32_t ph;
            const int s = stage_of(j, ph);
            ok = mbar_wait_bounded(&sh.full_b[s], ph);
            ok = ok && mbar_wait_bounded(&sh.full_a[j], (aphase >> j) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            aphase ^= 1u << j;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t dt = tm + abuf * PN32, ad = tm + TM_A + j * (SK / 2);
              const uint64_t desc = first + (uint64_t)(s * 2) * box;
              umma_f16_ts(dt, ad, desc, idesc, q == 0 ? 0u : 1u);
#pragma unroll
              for (int kk = 1; kk < 4; ++kk) umma_f16_ts(dt, ad + kk * 8, desc + kk * 2, idesc, 1u);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f16_ts(dt, ad + 32 + kk * 8, desc + box + kk * 2, idesc, 1u);
              umma_commit(&sh.empty_a[j]);
              if (part == PARTS - 1) umma_commit(&sh.empty_b[s]);
              if (q == PARTS * count - 1) umma_commit(&sh.acc_full[abuf]);
            }
            __syncwarp();
          }
          uint32_t ph;
          bstage = stage_of(count, ph);
          bphase = ph;
          cphase ^= 1u << abuf, abuf ^= 1u;
        }
      }
    }
    for (int t = cta; !FP32 && t < tiles && ok; t += ctas, abuf ^= 1) {
      for (int ks = ks0; ks < ks1 && ok; ++ks) {
        const int j = (ks - ks0) & 1;
        const bool fresh = ks == ks0, last = ks == ks1 - 1;
        ok = mbar_wait_bounded(&sh.full_a[j], (aphase >> j) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        aphase ^= 1u << j;
        issue(two ? 0u : abuf, j, fresh, last, !two);
        if (two && ok) issue(1u, j, fresh, last, true);
      }
    }
    if (!ok && lane == 0) many_timeout(a.status, sh);
    __syncwarp();
    if (elect_one()) {
      if constexpr (PAIR)
        umma_commit_pair_local(&sh.drain);
      else
        umma_commit(&sh.drain);
      (void)mbar_wait_bounded(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 2 && warp < 4) {
    // ---------------------------------------------------------------- codes to shared memory
    const int id = threadIdx.x - 64;
    const int64_t pitch = (int64_t)(a.p.d / 32) * BITS * 4;   // bytes per row
    const uint32_t ring = smem_u32(smem) + a.bstages * bstage_bytes;
    const int block_bytes = C::bytes(a.subs);
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = cta; t < tiles && ok; t += ctas) {
      const int64_t m0 = min(first_row(t), (int64_t)(a.nM - 1) * PM);
      const int rows = (int)min((int64_t)PM, a.p.r - m0);
      const char *q0 = reinterpret_cast<const char *>(a.p.qweight) + m0 * pitch;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded(&sh.empty_c[slot], phase ^ 1)) {
          if (lane == 0) many_timeout(a.status, sh);
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = ring + slot * block_bytes;
        const int k0 = kb * BCOLS;
        const int valid = min(BCOLS, a.p.d - k0) * BITS / 8;   // bytes of a row that exist
        const char *src = q0 + k0 * BITS / 8;
        // rows past the last and columns past the row are filled with zeros
        if (a.aligned) {
          if (id == 0) {
            mbar_arrive_expect_tx(&sh.full_c[slot], C::CODES);
#pragma unroll
            for (int x = 0; x < C::ROW; x += C::BOX)   // multiples of 16 bytes from multiples of 32 codes
              tma_load_2d(smem + a.bstages * bstage_bytes + slot * block_bytes + x * PM, &tmW,
                          kb * C::ROW + x, (int)m0, &sh.full_c[slot]);
          }
        } else {
          constexpr int PPR = C::ROW / 4;
#pragma unroll 4
          for (int i = 0; i < PM * PPR / LOADERS; ++i) {
            const int p = id + LOADERS * i, row = p / PPR, col = p % PPR * 4;
            const bool in = row < rows && col < valid;
            cp_async4(dst + C::place(row, col), in ? src + row * pitch + col : src, in ? 4 : 0);
          }
          if (id == 0) mbar_arrive(&sh.full_c[slot]);
        }
        for (int sub = 0; sub < a.subs; ++sub) {
          const int g = group_of(a, min(kb * (BCOLS / 32) + sub * (BCOLS / 32 / a.subs), a.p.d / 32 - 1));
          const uint32_t sz = dst + C::CODES + sub * (PM * 4);
#pragma unroll
          for (int i = 0; i < PM / LOADERS; ++i) {
            const int row = id + LOADERS * i;
            const int64_t at = (m0 + (row < rows ? row : 0)) * a.p.G + g;
            cp_async4(sz + row * 4, a.p.scales + at, row < rows ? 4 : 0);
            cp_async4(sz + a.subs * (PM * 4) + row * 4, a.p.zeros + at, row < rows ? 4 : 0);
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&sh.full_c[slot]))
                     : "memory");
        if (++slot == C::DEPTH) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 4 && warp < 4 + 4 * WGS) {
    // ---------------------------------------------------------------- weights to TMEM
    const int wg = (warp - 4) >> 2, quarter = warp & 3;
    const int as = wg / 2;                   // step of the block, A stage
    const int lrow = quarter * 32 + lane;
    const uint32_t ring = smem_u32(smem) + a.bstages * bstage_bytes;
    const int block_bytes = C::bytes(a.subs);
    // the parts of the block that this step's two 32-column chunks lie in
    const int sub0 = 2 * wg * a.subs / 8, sub1 = (2 * wg + 1) * a.subs / 8;
    int slot = 0, parity = 0;
    uint32_t phase = 0, aphase = 0, magic;
    asm volatile("mov.b32 %0, %1;" : "=r"(magic) : "n"(Pair<T>::M));
    bool ok = true;
    // (a warp that gave up still walks the tiles: the others wait for it at their barrier)
    for (int t = cta; t < tiles; t += ctas, parity ^= 1) {
      float inv = 1.f;
      if constexpr (HALF) {
        // the largest scale of each row over this CTA's columns: a warp takes
        // PM / (4 WGS) rows, lanes along the groups
        const int ga = group_of(a, ks0 * (SK / 32)), gb = group_of(a, min(ks1 * (SK / 32), a.p.d / 32) - 1);
        constexpr int EACH = PM / (4 * WGS);
        const int64_t m0 = first_row(t) + (warp - 4) * EACH;
        uint32_t top[EACH] = {};
        for (int g = ga + lane; g <= gb; g += 32) {
#pragma unroll
          for (int i = 0; i < EACH; ++i) {
            const int64_t row = m0 + i < a.p.r ? m0 + i : a.p.r - 1;
            top[i] = max(top[i], __float_as_uint(__ldg(a.p.scales + row * a.p.G + g)) & 0x7FFFFFFFu);
          }
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
          const uint32_t e = safe_exponent<BITS>(__reduce_max_sync(0xffffffffu, top[i]));
          if (lane == 0) sh.exponent[parity][(warp - 4) * EACH + i] = e;
        }
        // (the other parity's values were read before this barrier)
        asm volatile("bar.sync 1, %0;" ::"n"(128 * WGS) : "memory");
        inv = __uint_as_float((254u + LIFT<BITS> - sh.exponent[parity][lrow]) << 23);
      }
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        if (!mbar_wait_bounded(&sh.full_c[slot], phase)) {
          if (lane == 0) many_timeout(a.status, sh);
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (kb * BLK + as < ks1) {
          const uint32_t src = ring + slot * block_bytes;
          const int col = wg * (PK * BITS / 8);
          const uint32_t sz = ring + slot * block_bytes + C::CODES + lrow * 4;
          uint32_t w[2 * BITS];
          if constexpr (BITS == 3) {
#pragma unroll
            for (int i = 0; i < 6; i += 2)
              asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                           : "=r"(w[i]), "=r"(w[i + 1]) : "r"(src + C::place(lrow, col + i * 4)));
          } else {
#pragma unroll
            for (int i = 0; i < 2 * BITS; i += 4)
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                           : "r"(src + C::place(lrow, col + i * 4)));
          }
          float s;
          int z;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(sz + sub0 * (PM * 4)));
          asm volatile("ld.shared.s32 %0, [%1];" : "=r"(z) : "r"(sz + (a.subs + sub0) * (PM * 4)));
          uint32_t c0[16], c1[16];
          // 64 columns of this row to the A stage, when the MMAs have read the last ones
          auto hand_over = [&]() {
            if (!mbar_wait_bounded(&sh.empty_a[as], aphase ^ 1)) {
              if (lane == 0) many_timeout(a.status, sh);
              ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            tc_fence_after();
            const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + TM_A + wg * (PK / 2);
            tmem_st_x16(dst, c0);
            tmem_st_x16(dst + 16, c1);
            aphase ^= 1;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR)
                mbar_arrive_cluster(cluster_addr(&sh.full_a[as], 0));
              else
                mbar_arrive(&sh.full_a[as]);
            }
          };
          if constexpr (FP32) {
            auto zero = [](int z) { return __uint_as_float(0x4B000000u | (uint32_t)min(max(z, 0), (1 << BITS) - 1)); };
            const float sa = s * inv, za = zero(z);
            float sb = sa, zb = za;
            if (sub1 != sub0) {
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(sz + sub1 * (PM * 4)));
              asm volatile("ld.shared.s32 %0, [%1];" : "=r"(z) : "r"(sz + (a.subs + sub1) * (PM * 4)));
              sb = s * inv, zb = zero(z);
            }
            // (the words anew for each part, to the compiler: it would keep 64 numbers)
            auto renew = [&]() {
#pragma unroll
              for (int i = 0; i < 2 * BITS; ++i) asm volatile("" : "+r"(w[i]));
            };
            chunk_part<BITS, T, 0>(w, sa, za, c0);
            chunk_part<BITS, T, 0>(w + BITS, sb, zb, c1);
            hand_over();
            if (!ok) break;
            renew();
            chunk_part<BITS, T, 1>(w, sa, za, c0);
            chunk_part<BITS, T, 1>(w + BITS, sb, zb, c1);
            hand_over();
            if (!ok) break;
            if constexpr (PARTS == 3) {
              renew();
              chunk_part<BITS, T, 2>(w, sa, za, c0);
              chunk_part<BITS, T, 2>(w + BITS, sb, zb, c1);
              hand_over();
              if (!ok) break;
            }
          } else {
            Group<BITS, T> g;
            g.set(s * inv, z);
            chunk_weights<BITS, T>(w, g, magic, c0);
            if (sub1 != sub0) {
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(sz + sub1 * (PM * 4)));
              asm volatile("ld.shared.s32 %0, [%1];" : "=r"(z) : "r"(sz + (a.subs + sub1) * (PM * 4)));
              g.set(s * inv, z);
            }
            chunk_weights<BITS, T>(w + BITS, g, magic, c1);
            hand_over();
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive(&sh.empty_c[slot]);
        } else if (lane == 0) {
          mbar_arrive(&sh.empty_c[slot]);
        }
        if (++slot == C::DEPTH) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- results
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;
    uint32_t abuf = 0, cphase = 0;
    float *part = reinterpret_cast<float *>(smem);   // split k: [N][PM] sums of this CTA
    bool ok = true;
    for (int t = cta; t < tiles && ok; t += ctas, abuf ^= FP32 ? 0 : 1) {
      const int64_t row = first_row(t) + lrow;
      const bool live = row < a.p.r;
      float f = 1.f;
      if constexpr (HALF) {
        const float *srow = a.p.scales + (live ? row : a.p.r - 1) * a.p.G;
        const int ga = group_of(a, ks0 * (SK / 32)), gb = group_of(a, min(ks1 * (SK / 32), a.p.d / 32) - 1);
        uint32_t top = 0;
#pragma unroll 4
        for (int g = ga; g <= gb; ++g) top = max(top, __float_as_uint(__ldg(srow + g)) & 0x7FFFFFFFu);
        f = __uint_as_float((safe_exponent<BITS>(top) - LIFT<BITS>) << 23);
      }
      const float bias = a.p.bias && live ? load_as_float(a.p.bias, a.p.ytype, row) : 0.f;
      for (int h = 0; h < a.halves; ++h) {
        const uint32_t buf = a.halves == 2 ? h : abuf;
        // the tokens' scales, while the accumulator fills (a load per 16 tokens as they
        // were written took 5 us for 384 tokens)
        const int64_t t0 = ((int64_t)(t / nMt) * a.halves + h) * N;
        if (PAIR || a.ctas_k == 1) {
          __syncwarp();
          for (int c = lane; c < N; c += 32)
            sh.scale[quarter][c] = a.p.x_scales && t0 + c < a.p.n ? __ldg(a.p.x_scales + t0 + c) : 1.f;
          __syncwarp();
        }
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t base = lanes + (FP32 ? TM_SUM : buf * PN);
        if constexpr (FP32) {
          for (int kb = kb0; kb < kb1; ++kb, abuf ^= 1) {
            ok = mbar_wait_bounded(&sh.acc_full[abuf], (cphase >> abuf) & 1u);
            if (!ok && lane == 0) many_timeout(a.status, sh);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            cphase ^= 1u << abuf;
            tc_fence_after();
            add_sums(base, lanes + abuf * PN32, N, kb == kb0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[abuf]);
          }
          if (!ok) break;
        } else {
          ok = mbar_wait_bounded(&sh.acc_full[buf], (cphase >> buf) & 1u);
          if (!ok && lane == 0) many_timeout(a.status, sh);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          cphase ^= 1u << buf;
          tc_fence_after();
        }
        // tokens of this accumulator that exist
        const int count = (int)(a.p.n - t0 < N ? (a.p.n - t0 > 0 ? a.p.n - t0 : 0) : N);
        if (!PAIR && a.ctas_k > 1) {
          for (int c0 = 0; c0 < N; c0 += 16) {
            float v[16];
            tmem_ld_32x32b_x16(base + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c0 + i) * PM + lrow] = v[i] * f;
          }
        } else if constexpr (FP32) {
          settle |= write_tile<float>(base, count, f, bias, sh.scale[quarter], t0, row, a.p, sh.stage[quarter],
                                      lane);
        } else if (a.p.ytype == GPTQ_F16) {
          write_tile<__half>(base, count, f, bias, sh.scale[quarter], t0, row, a.p, sh.stage[quarter], lane);
        } else {
          write_tile<__nv_bfloat16>(base, count, f, bias, sh.scale[quarter], t0, row, a.p, sh.stage[quarter],
                                    lane);
        }
        tc_fence_before();
        __syncwarp();
        if (!FP32 && lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_cluster(cluster_addr(&sh.acc_empty[buf], 0));
          else
            mbar_arrive(&sh.acc_empty[buf]);
        }
      }
    }
  }

  __syncthreads();
  if (!PAIR && a.ctas_k > 1) {
    // one tile per cluster: add the CTAs' sums, each CTA its share of the tokens
    __syncwarp();
    cluster_sync();
    if (cta < tiles && !*(volatile int *)&sh.abort) {
      const float *part = reinterpret_cast<const float *>(smem);
      const int64_t m0 = (int64_t)(cta % a.nM) * PM, t0 = (int64_t)(cta / a.nM) * N;
      const int c0 = N * crank / a.ctas_k, c1 = N * (crank + 1) / a.ctas_k;
      // four rows of a token at a time, every CTA's share asked for before any is used
      for (int i = c0 * (PM / 4) + threadIdx.x; i < c1 * (PM / 4); i += MANY_THREADS) {
        const int64_t tok = t0 + i / (PM / 4), row = m0 + i % (PM / 4) * 4;
        if (tok >= a.p.n || row >= a.p.r) continue;
        float4 o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < a.ctas_k)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(o[k].x), "=f"(o[k].y), "=f"(o[k].z), "=f"(o[k].w)
                         : "r"(cluster_addr(part + i * 4, k)));
        }
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) y[0] += o[k].x, y[1] += o[k].y, y[2] += o[k].z, y[3] += o[k].w;
        const float s = a.p.x_scales ? __ldg(a.p.x_scales + tok) : 1.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          y[q] = fmaf(y[q], s, a.p.bias && row + q < a.p.r ? load_as_float(a.p.bias, a.p.ytype, row + q) : 0.f);
        const int64_t at = tok * a.p.r + row;
        if (!FP32 && a.p.r % 4 == 0 && reinterpret_cast<uintptr_t>(a.p.y) % 8 == 0) {
          uint2 w;
          if (a.p.ytype == GPTQ_F16) {
            const __half2 lo = __floats2half2_rn(y[0], y[1]), hi = __floats2half2_rn(y[2], y[3]);
            w = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
          } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(y[2], y[3]);
            w = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
          }
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.p.y) + at) = w;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (row + q < a.p.r) {
              store_float(a.p.y, a.p.ytype, at + q, y[q]);
              if constexpr (FP32) settle |= !(fabsf(y[q]) <= 3.402823466e38f);
            }
        }
      }
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_before();
  if constexpr (PAIR) {
    __syncwarp();
    cluster_sync();   // neither CTA's memory goes while the other may touch it
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
  if constexpr (FP32) {   // the results that this thread wrote, where no wait with a limit depends on it
    if (!settle) return;
    for (int t = cta; t < tiles; t += ctas) {
      const int64_t t0 = (int64_t)(t / nMt) * N, m0 = first_row(t);
      const bool split = a.ctas_k > 1;
      const int c0 = split ? N * crank / a.ctas_k : 0, c1 = split ? N * (crank + 1) / a.ctas_k : N;
      for (int i = c0 * PM + (split ? threadIdx.x * 4 : (warp & 3) * 32 + lane); i < c1 * PM;
           i += split ? MANY_THREADS * 4 : PM)
        for (int q = 0; q < (split ? 4 : 1); ++q) {
          const int64_t tok = t0 + i / PM, row = m0 + i % PM + q;
          if (tok < a.p.n && row < a.p.r) settle_result<BITS>(a.p, tok, row);
        }
    }
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

template <int BITS, typename T, bool PAIR, bool FP32>
int launch_kernel(const ManyArgs &a, const CUtensorMap &tx, const CUtensorMap &tw, int64_t ctas, int cluster,
                  size_t bytes, cudaStream_t st) {
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(packed_many_kernel<BITS, T, PAIR, FP32>, MANY_SMEM + 1024, attr)) return rc;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(MANY_THREADS);
  cfg.dynamicSmemBytes = bytes + 1024;
  cfg.stream = st;
  cfg.attrs = a.p.follows ? at : at + 1;
  cfg.numAttrs = (a.p.follows ? 1 : 0) + (cluster > 1 ? 1 : 0);
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, packed_many_kernel<BITS, T, PAIR, FP32>, tx, tw, a);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_last_error(__FILE__, __LINE__, "kernel launch", e);
    return GPTQ_ERR_CUDA;
  }
  return GPTQ_OK;
}

template <int BITS, typename T, bool FP32>
int launch_many(const PackedArgs &p, cudaStream_t st) {
  ManyArgs a{};
  a.p = p;
  const int sms = num_sms();
  const int64_t nM = (p.r + PM - 1) / PM;
  const int steps = (p.d + SK - 1) / SK;
  // Tokens per tile: all of them when they fit one accumulator; else pairs of CTAs,
  // and the width that wastes least.  A step of a tile takes its MMAs, about 4.7
  // clocks per token, or the conversion of its weights, about 1000 (both measured),
  // whichever is longer; two accumulators halve the conversions.  Where that leaves
  // most SMs idle, single CTAs that split k are faster: a step takes them about 1.2
  // times as long, and 14 steps go to start, fill and add up (pairs take ten).
  // Measured (pairs, single; us): 256 tokens, 4096 x 4096 26.1, 20.2; 4096 x 11008
  // 58.9, 37.3; 8192 x 8192 46.9, 51.8; 512 tokens, 4096 x 4096 27.1, 30.0.
  bool pair = p.n > PN && !FP32;
  int N = (int)((p.n + 15) / 16 * 16), halves = 1, ck = 1;
  if (pair) {
    int64_t best = INT64_MAX;
    for (int h = 1; h <= 2; ++h)
      for (int c = PN; c >= 96; c -= 32) {
        const int64_t pairs = (nM + 1) / 2 * ((p.n + c * h - 1) / (c * h));
        const int64_t rounds = (pairs + sms / 2 - 1) / (sms / 2), mma = c * h * 47 / 10;
        // (a round fills its pipeline again: 1000 tokens x 11008 x 4096, two rounds of 384
        // 86 us, three of 256 95)
        const int64_t cost = rounds * (steps * (mma > 1000 ? mma : 1000) + 3000) + 10000;
        if (cost < best) best = cost, N = c, halves = h;
      }
    // (7/8 of the SMs and clusters of four at most: larger ones do not all find room
    // at once; 256 tokens x 1024 x 4096 in 16 clusters of eight 24.6, of four 14.8)
    const int64_t parts = (p.n + PN - 1) / PN;
    for (int k = 2; k <= 4 && steps >= 2 * BLK * k && nM * parts * k <= sms * 7 / 8; ++k)
      if (((steps + k - 1) / k + 14) * 1200 < best) {
        best = ((steps + k - 1) / k + 14) * 1200;
        pair = false;
        N = (int)((p.n + parts * 16 - 1) / (parts * 16) * 16);
        halves = 1;
        ck = k;
      }
  }
  if constexpr (FP32) {
    // Tokens in equal parts, as many as take least, or split over k as below.
    const int64_t least = (p.n + PN32 - 1) / PN32;
    int64_t best = INT64_MAX;
    for (int64_t parts = least; parts <= 4 * least; ++parts) {
      const int c = (int)((p.n + parts * 16 - 1) / (parts * 16) * 16);
      const int64_t tiles = nM * ((p.n + c - 1) / c);
      if (const int64_t cost = (tiles + sms - 1) / sms * (steps + 10); cost < best) best = cost, N = c;
    }
  }
  const int64_t nMt = pair ? (nM + 1) / 2 : nM;
  const int64_t nN = (p.n + N * halves - 1) / (N * halves);
  if (nM * nN > INT32_MAX / 8) return GPTQ_ERR_INVALID_ARG;
  a.N = N;
  a.halves = halves;
  a.nM = (int)nM;
  a.nN = (int)nN;
  const int64_t tiles = nMt * nN;
  // k split over a cluster: the number of CTAs along it that takes least, a CTA
  // costing its steps and about ten more to start, fill and add up (at least two
  // blocks of codes each), of those whose clusters all find room at once: pairs on
  // every SM, up to four on 7/8 of them, eight on half (64 tokens x 2048 x 4096 as 16
  // clusters of eight 20.9 us, of four 13.1)
  if (FP32 || p.n <= PN) {
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 8 && (c == 1 || steps >= 2 * BLK * c); ++c) {
      if (c > 1 && tiles * c > (c == 2 ? sms : c <= 4 ? sms * 7 / 8 : sms / 2)) break;
      // (one CTA walks several tiles without starting again; a split one does not)
      const int64_t rounds = (tiles + sms - 1) / sms, each = (steps + c - 1) / c;
      const int64_t cost = c == 1 ? rounds * each + 10 : each + 12;
      if (cost < best) best = cost, ck = c;
    }
  }
  a.ctas_k = ck;
  const int stage = (pair ? N / 2 : N) * SK * 2;
  using C = CodeBlock<BITS>;
  a.subs = p.group < 0 || p.group % 256 == 0 ? 1 : p.group % 128 == 0 ? 2 : p.group % 64 == 0 ? 4 : 8;
  const size_t codes = (size_t)C::DEPTH * C::bytes(a.subs);
  const int nb = (int)((MANY_SMEM - codes) / stage);
  static_assert((MANY_SMEM - (size_t)C::DEPTH * C::bytes(8)) / (PN * SK * 2) >= 2,
                "too few stages of x");
  a.bstages = nb > MAXB ? MAXB : nb;
  // (the sums of a split k, N PM floats, take the place of two stages of x)
  const size_t bytes = (size_t)a.bstages * stage + codes;
  a.aligned = reinterpret_cast<uintptr_t>(p.qweight) % 16 == 0 &&
              ((int64_t)(p.d / 32) * BITS) % 4 == 0;
  a.gdiv = p.group > 0 ? (uint32_t)(((1ull << 31) + p.group / 32 - 1) / (p.group / 32)) : 0;
  a.status = device_status_word();
  if (!a.status) return GPTQ_ERR_CUDA;
  EncodeTiledFn enc = encode_fn();
  CUtensorMap tx;
  const cuuint64_t gdim[2] = {(cuuint64_t)p.d, (cuuint64_t)p.n};
  const cuuint64_t gstride[1] = {(cuuint64_t)p.d * 2};
  const cuuint32_t box[2] = {(cuuint32_t)PK, (cuuint32_t)(pair ? N / 2 : N)};
  const cuuint32_t es[2] = {1, 1};
  if (!enc || enc(&tx, Pair<T>::M == 0x64006400u ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  2, const_cast<void *>(p.x), gdim, gstride, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    set_last_error_msg(__FILE__, __LINE__, "cuTensorMapEncodeTiled rejected the activations");
    return GPTQ_ERR_CUDA;
  }
  // codes as bytes; rows on 16-byte boundaries
  CUtensorMap tw = tx;
  if (a.aligned) {
    const cuuint64_t wdim[2] = {(cuuint64_t)p.d * BITS / 8, (cuuint64_t)p.r};
    const cuuint64_t wstride[1] = {(cuuint64_t)p.d * BITS / 8};
    const cuuint32_t wbox[2] = {(cuuint32_t)C::BOX, (cuuint32_t)PM};
    if (enc(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint32_t *>(p.qweight), wdim, wstride,
            wbox, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            BITS == 3 ? CU_TENSOR_MAP_SWIZZLE_NONE
                      : (C::BOX == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B),
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
      set_last_error_msg(__FILE__, __LINE__, "cuTensorMapEncodeTiled rejected the packed weights");
      return GPTQ_ERR_CUDA;
    }
  }
  if constexpr (!FP32)
    if (pair)
      return launch_kernel<BITS, T, true, false>(a, tx, tw, 2 * (tiles < sms / 2 ? tiles : sms / 2), 2, bytes, st);
  return launch_kernel<BITS, T, false, FP32>(a, tx, tw, ck > 1 ? tiles * ck : (tiles < sms ? tiles : sms), ck,
                                             bytes, st);
}

template <typename T, bool FP32>
int launch_many_type(const PackedArgs &p, cudaStream_t st) {
  switch (p.bits) {
    case 2: return launch_many<2, T, FP32>(p, st);
    case 3: return launch_many<3, T, FP32>(p, st);
    case 4: return launch_many<4, T, FP32>(p, st);
    default: return launch_many<8, T, FP32>(p, st);
  }
}

}  // namespace
}  // namespace gptq
