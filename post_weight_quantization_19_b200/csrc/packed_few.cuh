// gptq_packed_linear for few tokens: y = x W^^T + bias, bound by reading the
// packed weights once (r d bits/8 + 8 r G bytes) and by the instructions that
// take the codes out of their words.
//
// A warp multiplies 32 rows of codes (two m16 tiles) with up to 8 or 16
// tokens on warp-level matrix instructions (mma.sync), whose operands come from
// registers: a code goes from its packed word to an operand in about one
// instruction, with nothing written back to shared or tensor memory on the way.
// (mma.sync reaches a quarter of tcgen05's rate: 0.46 m16n8k16 per clock and SM
// measured.  For few tokens that is enough: turning codes into operands takes longer.)
//
// The order of k inside a matrix instruction is free as long as both operands
// agree.  A thread takes eight codes of a row at a time (a unit): one 32-bit
// word of 4-bit codes.  Where a group covers the 128 columns of a stage, thread
// t of a row's four takes the units of the 32-column chunk t, which it reads at
// once; smaller groups need all four threads inside one chunk, so thread t takes
// unit t of every chunk (FINE).
//
// 16-bit x: the operand is B + q, whose bits are the code's bits and a constant:
//   fp16: B = 0, the code as a subnormal number in its upper bits, q 2^(2 bits - 34)
//         (8-bit codes q 2^-24; exact, and so are its products in fp32); every second
//         code stays one place higher, 2^bits times that, and is summed apart, which
//         saves a shift.  (The tensor core aligns products by their exponents, a
//         subnormal number's as if it were 2^-14, and drops what lies 25 bits
//         below: codes in the lowest bits, and sum x from ones of 2^-24, left sums good
//         to 2^-17.  12288 x 49152, one token: 90.3 us so, 93.5 with codes in the upper bits);
//   bf16: B = 16 or 4 for 4- or 2-bit codes, the code in the upper mantissa
//         bits; 3-bit codes B = 64 and 8 in turn, at two places of the mantissa,
//         which saves two shifts of four.  (8-bit codes do not fit: q - z
//         through fp32 instead.)
// and one more product with a matrix of ones gives sum x (for each B), so that a
// group adds
//   s (sum (B + q) x - (B + z) sum x).
// The terms that cancel are at most (B + q + z) / |q - z| times what q - z itself
// would sum, held in fp32; results that are no numbers for it (infinities in x) are
// formed again from q - z (settle_lost).  8-bit x: q and x as integers, sums exact.
//
// Each warp runs its own ring of cp.async stages of 128 columns (weights, x,
// scales, zeros) and meets the others only at the end: the k range is split
// over the CTA's warps and over a cluster of CTAs, whose partial sums are added
// through distributed shared memory in a fixed order.
//
// Measured, one token, inputs from HBM: 12288 x 49152, 3 bits, bf16 129 us (2.1 TB/s; the
// integer pipe is busy 65 % of the time, 2.3 instructions per clock); 4 bits, fp16 94 us
// (3.6 TB/s); 4096 x 4096, 4 bits 5.9 us, most of it launch, fill and the last sums; 11008
// x 4096 with 8-bit x 10.5 us.
#pragma once

#include "packed_linear.h"

namespace gptq {
namespace {

constexpr int KS = 128;        // columns per stage
constexpr int ROWS = 32;       // rows per warp (two m16 tiles)

template <int BITS, int XT, int NT, bool FINE>
struct Few {
  static constexpr bool INT8 = XT == GPTQ_I8;
  // 8-bit codes with bf16: operands q - z
  static constexpr bool EXACT = BITS == 8 && XT == GPTQ_BF16;
  // fp16 codes of fewer bits: the pairs at odd places are summed apart
  static constexpr bool TWO = BITS != 8 && XT == GPTQ_F16;
  // bf16 codes of 3 bits: two bases
  static constexpr bool BASES = BITS == 3 && XT == GPTQ_BF16;
  // Row strides in shared memory, chosen so that the rows a warp reads at once
  // fall on different banks.
  static constexpr int WSTRIDE = FINE ? (BITS == 4 ? 80 : BITS == 8 ? 160 : 48)
                                      : (BITS == 4 ? 64 : BITS == 8 ? 144 : BITS == 3 ? 48 : 32);
  static constexpr int XB = INT8 ? 1 : 2;                         // bytes of an element of x
  static constexpr int XROW = KS * XB;
  static constexpr int XSTRIDE = INT8 ? (FINE ? 160 : 144) : 320;
  static constexpr int WBYTES = ROWS * WSTRIDE;
  static constexpr int STAGES = NT == 2 && BITS == 8 ? 2 : 3;
  // Scales and zeros: FINE, those of a stage's four chunks lie in the stage; else
  // blocks of four groups in slots of the warp's own, so that a 32-byte
  // sector is fetched twice and not for every stage (which doubled the traffic
  // from L2: 121 us instead of 81 for 12288 x 49152, 4 bits).
  static constexpr int SZBYTES = FINE ? ROWS * 4 * 4 * 2 : 0;
  static constexpr int SZSLOT = ROWS * 4 * 4 * 2;
  static constexpr int SZSLOTS = STAGES + 1;   // one per stage in flight, at worst, and the last one's
  static constexpr int SZWARP = FINE ? 0 : SZSLOTS * SZSLOT;
  __host__ __device__ static constexpr int stage_bytes(int tokens) {
    return (WBYTES + SZBYTES + tokens * XSTRIDE + 127) / 128 * 128;
  }
  static constexpr int MAX_WARPS = 16;                            // of a CTA: 8, 12 or 16
};
constexpr size_t FEW_SMEM = 226 * 1024;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Reads of the ring: plain loads, which the compiler may move among the products
// but not over the waits.  `a` is an address in shared memory's window.
template <typename V>
__device__ __forceinline__ V lds(uint32_t a) {
  return *reinterpret_cast<const V *>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) { return lds<uint32_t>(a); }
__device__ __forceinline__ uint32_t lds16(uint32_t a) { return lds<uint16_t>(a); }
__device__ __forceinline__ uint2 lds64(uint32_t a) { return lds<uint2>(a); }
__device__ __forceinline__ uint4 lds128(uint32_t a) { return lds<uint4>(a); }

// d = a b (+ d): with FIRST the sum starts here.
template <int XT, bool FIRST>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  const float z = 0.f;
  if constexpr (FIRST) {
    if constexpr (XT == GPTQ_F16)
      asm(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%10,%10,%10,%10};"
          : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
    else
      asm(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%10,%10,%10,%10};"
          : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
  } else {
    if constexpr (XT == GPTQ_F16)
      asm(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
      asm(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}
template <bool FIRST>
__device__ __forceinline__ void mma8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
  else
    asm(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A row's share of a stage, from shared memory: the four units of chunk t, or
// (FINE) unit t of the four chunks; each as it lies in the stream (8-bit codes:
// two words), low bits first, anything above.
template <int BITS, bool FINE>
__device__ __forceinline__ void row_units(uint32_t row, int t, uint2 (&u)[4]) {
  if constexpr (FINE) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (BITS == 4) u[c].x = lds32(row + c * 16 + t * 4);
      if constexpr (BITS == 2) u[c].x = lds16(row + c * 8 + t * 2);
      if constexpr (BITS == 8) u[c] = lds64(row + c * 32 + t * 8);
      if constexpr (BITS == 3) {   // 24 bits from bit 24 t of the chunk's 96
        const int at = (t * 24) >> 5;
        const uint32_t lo = lds32(row + c * 12 + at * 4);
        const uint32_t hi = lds32(row + c * 12 + min(at + 1, 2) * 4);
        u[c].x = __funnelshift_r(lo, hi, (t * 24) & 31);
      }
    }
  } else {
    if constexpr (BITS == 4) {
      const uint4 v = lds128(row + t * 16);
      u[0].x = v.x, u[1].x = v.y, u[2].x = v.z, u[3].x = v.w;
    }
    if constexpr (BITS == 2) {
      const uint2 v = lds64(row + t * 8);
      u[0].x = v.x, u[1].x = v.x >> 16, u[2].x = v.y, u[3].x = v.y >> 16;
    }
    if constexpr (BITS == 8) {
      const uint4 v = lds128(row + t * 32), w = lds128(row + t * 32 + 16);
      u[0] = make_uint2(v.x, v.y), u[1] = make_uint2(v.z, v.w);
      u[2] = make_uint2(w.x, w.y), u[3] = make_uint2(w.z, w.w);
    }
    if constexpr (BITS == 3) {
      const uint32_t a = lds32(row + t * 12), b = lds32(row + t * 12 + 4), c = lds32(row + t * 12 + 8);
      u[0].x = a;
      u[1].x = __funnelshift_r(a, b, 24);
      u[2].x = __funnelshift_r(b, c, 16);
      u[3].x = c >> 8;
    }
  }
}

// B of the operand B + q (bf16), see above; 3-bit codes: of the even pairs.
template <int BITS, int XT>
constexpr float operand_base() {
  return XT == GPTQ_BF16 && BITS != 8 ? (BITS == 4 ? 16.f : BITS == 3 ? 64.f : 4.f) : 0.f;
}

// fp16: what a code of 1 stands for (the first of each two, code_pairs).
template <int BITS>
constexpr float CODE_UNIT = BITS == 8 ? 0x1p-24f : BITS == 4 ? 0x1p-22f : BITS == 3 ? 0x1p-20f : 0x1p-18f;

// A zero point, clamped to the codes, as its group uses it: itself for 8-bit x, 2^23
// + z for 8-bit codes with bf16, else -(B + z) in units of the operands' codes (as
// float bits).
template <int BITS, int XT>
__device__ __forceinline__ uint32_t prepare_zero(uint32_t raw) {
  const uint32_t z = (uint32_t)min(max((int)raw, 0), (1 << BITS) - 1);
  if constexpr (XT == GPTQ_I8) return z;
  const float f = __uint_as_float(0x4B000000u | z);   // 2^23 + z
  if constexpr (BITS == 8 && XT == GPTQ_BF16) return __float_as_uint(f);
  const float v = (8388608.f - operand_base<BITS, XT>()) - f;
  return __float_as_uint(XT == GPTQ_F16 ? v * CODE_UNIT<BITS> : v);
}

// The eight codes of a unit as four pairs of operands: (0,4), (1,5), (2,6),
// (3,7), or for 8-bit codes (0,1), (2,3), (4,5), (6,7); fp16 codes of fewer
// bits: the second and fourth pair times 2^BITS.  zf = 2^23 + z, for 8-bit
// codes with bf16 only.  base: the bits of the operands' B (bf16), of the even and
// the odd pairs, in registers that the compiler does not see through, so that
// mask and base take one instruction (which holds one constant).
template <int BITS, int XT>
__device__ __forceinline__ void code_pairs(uint2 w, float zf, const uint32_t (&base)[2],
                                           uint32_t (&o)[4]) {
  if constexpr (BITS == 8) {
    if constexpr (XT == GPTQ_F16) {
      o[0] = __byte_perm(w.x, 0, 0x4140), o[1] = __byte_perm(w.x, 0, 0x4342);
      o[2] = __byte_perm(w.y, 0, 0x4140), o[3] = __byte_perm(w.y, 0, 0x4342);
    } else {
      // 8 bits do not fit bf16's mantissa beside a base: through fp32, whose upper
      // half holds |q - z| <= 255 exactly
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = i < 2 ? w.x : w.y;
        const float a = __uint_as_float(__byte_perm(v, 0x4B000000u, (i & 1) ? 0x7442 : 0x7440)) - zf;
        const float b = __uint_as_float(__byte_perm(v, 0x4B000000u, (i & 1) ? 0x7443 : 0x7441)) - zf;
        o[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
      }
    }
  } else {
    // codes 0..3 to the low half, 4..7 to the high half, code i at bit i BITS
    uint32_t v = w.x;
    if constexpr (BITS == 3) v = (v & 0x0000FFFFu) | ((v << 4) & 0xFFFF0000u);
    if constexpr (BITS == 2) v = __byte_perm(v, 0, 0x4140);
    constexpr uint32_t mask = ((1u << BITS) - 1u) * 0x00010001u;
    if constexpr (XT == GPTQ_F16) {
      constexpr int P = 10 - 2 * BITS, R = 2 * BITS - P;
      const uint32_t u = v << P, h = R > 0 ? v >> (R > 0 ? R : 0) : v << (R < 0 ? -R : 0);
      o[0] = u & (mask << P), o[1] = u & (mask << (P + BITS));
      o[2] = h & (mask << P), o[3] = h & (mask << (P + BITS));
    } else if constexpr (BITS == 3) {
      // codes 0 and 2 at bit 1 (64 + q), 1 and 3 at bit 4 (8 + q)
      const uint32_t u = v << 1, h = v >> 5;
      o[0] = (u & 0x000E000Eu) | base[0], o[1] = (u & 0x00700070u) | base[1];
      o[2] = (h & 0x000E000Eu) | base[0], o[3] = (h & 0x00700070u) | base[1];
    } else {
      // at bit P, the top of the mantissa: exponent of 2^BITS
      constexpr int P = 7 - BITS;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int left = P - BITS * i;
        const uint32_t u = left > 0 ? v << (left > 0 ? left : 0) : v >> (left < 0 ? -left : 0);
        o[i] = (u & (mask << P)) | base[0];
      }
    }
  }
}

// The eight codes as bytes: {0, 2, 4, 6}, {1, 3, 5, 7} for 4-bit codes, else
// in order.
template <int BITS>
__device__ __forceinline__ uint2 code_bytes(uint2 w) {
  if constexpr (BITS == 8) {
    return w;
  } else if constexpr (BITS == 4) {
    return make_uint2(w.x & 0x0F0F0F0Fu, (w.x >> 4) & 0x0F0F0F0Fu);
  } else {
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
}

struct FewArgs {
  PackedArgs p;
  int ctas_k;        // CTAs of a cluster, along k
  int stage_bytes;   // of one stage of one warp
  int aligned;       // rows of codes start on 16-byte boundaries
  int sz_aligned;    // rows of scales and zeros too, in whole fours
  uint32_t gdiv;     // ceil(2^31 / (group / 32)), 0 for one group
};

// A thread's results that are no numbers again, from their definition, after its last
// tile.  A function of its own, with its arguments by value: as part of the kernel, in
// or behind the loop over the tiles, it cost every call 4 to 14 % (12288 x 49152, 3 bits,
// one token: 128 us, 134 to 146).  A thread takes a result, so a token with an infinity
// costs milliseconds on the largest layers.
template <int BITS, int NT>
__device__ __noinline__ void settle_lost(const FewArgs a, int crank, int cta, int ctas) {
  constexpr int CELLS = ROWS * 8 * NT;
  const int per = CELLS / a.ctas_k, first = crank * per;
  const int64_t tok0 = (int64_t)blockIdx.y * (8 * NT);
  for (int64_t row0 = (int64_t)cta * ROWS; row0 < a.p.r; row0 += (int64_t)ctas * ROWS)
    for (int i = first + threadIdx.x; i < first + per; i += blockDim.x) {
      const int64_t tok = tok0 + i / ROWS, row = row0 + i % ROWS;
      if (tok >= a.p.n || row >= a.p.r) continue;
      if (fabsf(load_as_float(a.p.y, a.p.ytype, tok * a.p.r + row)) <= 3.402823466e38f) continue;
      float v = sum_in_64_bits<BITS>(a.p, tok, row);
      if (a.p.bias) v += load_as_float(a.p.bias, a.p.ytype, row);
      store_float(a.p.y, a.p.ytype, tok * a.p.r + row, v);
    }
}

template <int BITS, int XT, int NT, bool FINE>
__global__ void __launch_bounds__(32 * Few<BITS, XT, NT, FINE>::MAX_WARPS)
    packed_few_kernel(const FewArgs a) {
  using F = Few<BITS, XT, NT, FINE>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int crank = blockIdx.x % a.ctas_k;
  const int64_t tok0 = (int64_t)blockIdx.y * (8 * NT);
  const int ntok = (int)min((int64_t)(8 * NT), a.p.n - tok0);
  const int d = a.p.d;
  // this warp's stages of every tile
  const int total = (d + KS - 1) / KS;
  const int parts = a.ctas_k * warps, part_id = crank * warps + warp;
  const int s0 = total * part_id / parts, s1 = total * (part_id + 1) / parts;
  const int tiles = (int)((a.p.r + ROWS - 1) / ROWS);
  const int cta = blockIdx.x / a.ctas_k, ctas = gridDim.x / a.ctas_k;

  const uint32_t ring = smem_u32(smem) + warp * (F::STAGES * a.stage_bytes + F::SZWARP);
  const uint32_t sz_ring = ring + F::STAGES * a.stage_bytes;
  const int pitch = d / 32 * BITS * 4;            // bytes per row
  // The loading cursor: stage ls of tile lt.  It runs ahead of the computing one
  // into the CTA's next tile, so that no tile starts with an empty ring.  What
  // a thread copies keeps its place from stage to stage: 16-byte piece lane +
  // 32 i of the rows of codes, and of the tokens.
  constexpr int PIECES = F::XROW / 16;             // of a token
  int lt = cta, ls = s0;
  const char *wsrc = nullptr;
  int woff[BITS];
  int64_t szrow = 0;
  const int xtok = lane / PIECES, xpiece = lane % PIECES;
  // (16-bit x of a coarse stage as [unit][chunk])
  const int xat = !F::INT8 && !FINE ? (xpiece & 3) * 4 + (xpiece >> 2) : xpiece;
  const char *xsrc = reinterpret_cast<const char *>(a.p.x) + (tok0 + xtok) * d * F::XB + xpiece * 16;
  auto open_tile = [&]() {
    const int64_t row0 = (int64_t)lt * ROWS;
    const int last = (int)min((int64_t)ROWS, a.p.r - row0) - 1;   // rows past it: its codes again, dropped
    wsrc = reinterpret_cast<const char *>(a.p.qweight) + row0 * pitch;
#pragma unroll
    for (int i = 0; i < BITS; ++i) {
      const int p = lane + 32 * i;
      woff[i] = min(p / BITS, last) * pitch + p % BITS * 16;
    }
    szrow = (row0 + min(lane, last)) * a.p.G;
  };

  auto group_of = [&](int chunk) { return (int)(((uint64_t)(uint32_t)chunk * a.gdiv) >> 31); };
  int sz_block = -1, sz_slot = 0;   // the last block of four groups asked for, its slot
  auto issue = [&](int slot) {
    if (lt >= tiles || s0 >= s1) return;
    if (ls == s0) {
      open_tile();
      sz_block = -1;
    }
    const int s = ls, tile = lt;
    if (++ls == s1) ls = s0, lt += ctas;
    const uint32_t base = ring + slot * a.stage_bytes;
    const int k0 = s * KS, cols = min(KS, d - k0);
    const char *w = wsrc + s * (KS * BITS / 8);
    if (a.aligned && cols == KS) {
#pragma unroll
      for (int i = 0; i < BITS; ++i) {
        const int p = lane + 32 * i;
        cp_async16(base + p / BITS * F::WSTRIDE + p % BITS * 16, w + woff[i], 16);
      }
    } else {
      const int bytes = cols * BITS / 8;             // of a row
      const int last = (int)min((int64_t)ROWS, a.p.r - (int64_t)tile * ROWS) - 1;
#pragma unroll 4
      for (int i = 0; i < 4 * BITS; ++i) {
        const int p = lane + 32 * i, row = p / (4 * BITS), col = p % (4 * BITS) * 4;
        const bool in = col < bytes;
        cp_async4(base + row * F::WSTRIDE + col, w + (min(row, last) * pitch + (in ? col : 0)),
                  in ? 4 : 0);
      }
    }
    // scales and zeros: lane = row
    if constexpr (FINE) {
      const uint32_t sz = base + F::WBYTES + lane * 16;
      if (a.sz_aligned && a.p.group == 32) {
        cp_async16(sz, a.p.scales + szrow + s * 4, 16);
        cp_async16(sz + ROWS * 16, a.p.zeros + szrow + s * 4, 16);
      } else {   // the stage's groups, one behind the other: two but for rows of odd alignment
        const int g0 = group_of(s * 4), g1 = group_of(min(s * 4 + 3, d / 32 - 1));
        if (a.sz_aligned && (g0 & 1) == 0 && g1 <= g0 + 1) {
          cp_async8(sz, a.p.scales + szrow + g0);
          cp_async8(sz + ROWS * 16, a.p.zeros + szrow + g0);
        } else {
          for (int gi = g0; gi <= g1; ++gi) {
            cp_async4(sz + (gi - g0) * 4, a.p.scales + szrow + gi, 4);
            cp_async4(sz + ROWS * 16 + (gi - g0) * 4, a.p.zeros + szrow + gi, 4);
          }
        }
      }
    } else {
      const int block = group_of(s * 4) >> 2;
      if (block != sz_block) {
        sz_block = block;
        sz_slot = sz_slot + 1 == F::SZSLOTS ? 0 : sz_slot + 1;
        const uint32_t sz = sz_ring + sz_slot * F::SZSLOT + lane * 16;
        if (a.sz_aligned) {
          cp_async16(sz, a.p.scales + szrow + block * 4, 16);
          cp_async16(sz + ROWS * 16, a.p.zeros + szrow + block * 4, 16);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int gi = min(block * 4 + c, a.p.G - 1);
            cp_async4(sz + c * 4, a.p.scales + szrow + gi, 4);
            cp_async4(sz + ROWS * 16 + c * 4, a.p.zeros + szrow + gi, 4);
          }
        }
      }
    }
    // x
    const bool in = xpiece * 16 < cols * F::XB;
    const char *x = xsrc + (int64_t)k0 * F::XB - (in ? 0 : xpiece * 16);
    uint32_t xdst = base + F::WBYTES + F::SZBYTES + xtok * F::XSTRIDE + xat * 16;
    for (int tok = xtok; tok < ntok; tok += 32 / PIECES) {
      cp_async16(xdst, x, in ? 16 : 0);
      x += (int64_t)d * (32 / PIECES * F::XB);
      xdst += 32 / PIECES * F::XSTRIDE;
    }
  };

  if (a.p.follows) asm volatile("griddepcontrol.wait;" ::: "memory");   // x
#pragma unroll
  for (int i = 0; i < F::STAGES - 1; ++i) {
    issue(i);
    cp_commit();
  }
  // The matrix of ones, as values the compiler does not see through: it would set four
  // registers anew for every product.
  uint32_t ones[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("mov.b32 %0, %1;"
                 : "=r"(ones[i])
                 : "n"(XT == GPTQ_F16 ? 0x3C003C00 : XT == GPTQ_BF16 ? 0x3F803F80 : 0x01010101));
  // bf16: 2^BITS at the top of the mantissa; 3-bit codes 64 and 8 (code_pairs)
  uint32_t bases[2];
  asm volatile("mov.b32 %0, %1;"
               : "=r"(bases[0])
               : "n"(BITS == 3 ? 0x42804280 : ((127 + BITS) << 7) * 0x00010001));
  asm volatile("mov.b32 %0, %1;" : "=r"(bases[1]) : "n"(0x41004100));
  // tokens past the last: its values again (their columns are dropped)
  uint32_t xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xrow[j] = min(j * 8 + g, ntok - 1) * F::XSTRIDE;
  int slot = 0, cslot = 0;
  // [warps][COLS][ROWS]
  float *red = reinterpret_cast<float *>(smem + warps * (F::STAGES * a.stage_bytes + F::SZWARP));
  bool lost = false;   // a result of this thread's is not a number's
  for (int tile = cta; tile < tiles; tile += ctas) {
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;
    int cblock = -1;   // as sz_block, of the computing cursor
    for (int s = s0; s < s1; ++s) {
      cp_wait<F::STAGES - 2>();
      __syncwarp();
      {
        int ns = slot + F::STAGES - 1;
        if (ns >= F::STAGES) ns -= F::STAGES;
        issue(ns);
        cp_commit();
      }
      const uint32_t base = ring + slot * a.stage_bytes;
      const uint32_t xbase = base + F::WBYTES + F::SZBYTES;
      // scales of rows 0, 1, ... of this stage's (first) group, 16 bytes apart; zeros behind
      uint32_t sz = base + F::WBYTES;
      if constexpr (!FINE) {
        const int gi = group_of(s * 4);
        if (gi >> 2 != cblock) {
          cblock = gi >> 2;
          cslot = cslot + 1 == F::SZSLOTS ? 0 : cslot + 1;
          // the block's zero points, made ready by the lane of their row
          const uint32_t at = sz_ring + cslot * F::SZSLOT + ROWS * 16 + lane * 16;
          uint4 z = lds128(at);
          z.x = prepare_zero<BITS, XT>(z.x), z.y = prepare_zero<BITS, XT>(z.y);
          z.z = prepare_zero<BITS, XT>(z.z), z.w = prepare_zero<BITS, XT>(z.w);
          *reinterpret_cast<uint4 *>(__cvta_shared_to_generic(at)) = z;
          __syncwarp();
        }
        sz = sz_ring + cslot * F::SZSLOT + (gi & 3) * 4;
      }
      uint32_t sub[4] = {};   // FINE: where the chunks' groups lie
      if constexpr (FINE) {
        const int g0 = group_of(s * 4);
#pragma unroll
        for (int u = 1; u < 4; ++u) sub[u] = (group_of(min(s * 4 + u, d / 32 - 1)) - g0) * 4;
      }
      uint2 lo[2][4], hi[2][4];   // rows g and g + 8 of the two tiles
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        row_units<BITS, FINE>(base + (m * 16 + g) * F::WSTRIDE, t, lo[m]);
        row_units<BITS, FINE>(base + (m * 16 + 8 + g) * F::WSTRIDE, t, hi[m]);
      }
      float part[2][NT][4], odd[2][NT][4], sx[NT][4], sx2[NT][4];
      int ipart[2][NT][4], isx[NT][4];
      float zf[2][2] = {};
      auto zero_point = [&](int m, int h, int u) {
        const uint32_t z = lds32(sz + ROWS * 16 + (m * 16 + h * 8 + g) * 16 + sub[u]);
        return FINE ? prepare_zero<BITS, XT>(z) : z;
      };
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool first = FINE || u == 0;   // a sum starts with this unit
        if constexpr (!F::INT8) {
          if (F::EXACT && first) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) zf[m][h] = __uint_as_float(zero_point(m, h, u));
          }
          // which pairs share a product: one choice for the codes and the ones, or x
          // would be copied into other register pairs
          constexpr int B1 = F::TWO || F::BASES ? 2 : 1, B2 = F::TWO || F::BASES ? 1 : 2;
          uint32_t xb[NT][4];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            // (a coarse stage: piece t of unit u; FINE: piece t of chunk u -- the same place)
            const uint4 v = lds128(xbase + xrow[j] + u * 64 + t * 16);
            if constexpr (BITS == 8) {
              xb[j][0] = v.x, xb[j][1] = v.y, xb[j][2] = v.z, xb[j][3] = v.w;
            } else {
              xb[j][0] = __byte_perm(v.x, v.z, 0x5410), xb[j][1] = __byte_perm(v.x, v.z, 0x7632);
              xb[j][2] = __byte_perm(v.y, v.w, 0x5410), xb[j][3] = __byte_perm(v.y, v.w, 0x7632);
            }
            if constexpr (!F::EXACT) {
              if constexpr (F::BASES) {
                if (first) {
                  mma16<XT, true>(sx[j], ones[0], ones[1], ones[2], ones[3], xb[j][0], xb[j][2]);
                  mma16<XT, true>(sx2[j], ones[0], ones[1], ones[2], ones[3], xb[j][1], xb[j][3]);
                } else {
                  mma16<XT, false>(sx[j], ones[0], ones[1], ones[2], ones[3], xb[j][0], xb[j][2]);
                  mma16<XT, false>(sx2[j], ones[0], ones[1], ones[2], ones[3], xb[j][1], xb[j][3]);
                }
              } else {
                if (first)
                  mma16<XT, true>(sx[j], ones[0], ones[1], ones[2], ones[3], xb[j][0], xb[j][B1]);
                else
                  mma16<XT, false>(sx[j], ones[0], ones[1], ones[2], ones[3], xb[j][0], xb[j][B1]);
                mma16<XT, false>(sx[j], ones[0], ones[1], ones[2], ones[3], xb[j][B2], xb[j][3]);
              }
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t pl[4], ph[4];
            code_pairs<BITS, XT>(lo[m][u], zf[m][0], bases, pl);
            code_pairs<BITS, XT>(hi[m][u], zf[m][1], bases, ph);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              if constexpr (F::TWO) {
                if (first) {
                  mma16<XT, true>(part[m][j], pl[0], ph[0], pl[2], ph[2], xb[j][0], xb[j][2]);
                  mma16<XT, true>(odd[m][j], pl[1], ph[1], pl[3], ph[3], xb[j][1], xb[j][3]);
                } else {
                  mma16<XT, false>(part[m][j], pl[0], ph[0], pl[2], ph[2], xb[j][0], xb[j][2]);
                  mma16<XT, false>(odd[m][j], pl[1], ph[1], pl[3], ph[3], xb[j][1], xb[j][3]);
                }
              } else {
                if (first)
                  mma16<XT, true>(part[m][j], pl[0], ph[0], pl[B1], ph[B1], xb[j][0], xb[j][B1]);
                else
                  mma16<XT, false>(part[m][j], pl[0], ph[0], pl[B1], ph[B1], xb[j][0], xb[j][B1]);
                mma16<XT, false>(part[m][j], pl[B2], ph[B2], pl[3], ph[3], xb[j][B2], xb[j][3]);
              }
            }
          }
        } else {
          uint32_t xb[NT][2];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint2 v = lds64(xbase + xrow[j] + (FINE ? u * 32 + t * 8 : t * 32 + u * 8));
            if constexpr (BITS == 4) {
              xb[j][0] = __byte_perm(v.x, v.y, 0x6420), xb[j][1] = __byte_perm(v.x, v.y, 0x7531);
            } else {
              xb[j][0] = v.x, xb[j][1] = v.y;
            }
            if (first)
              mma8<true>(isx[j], ones[0], ones[1], ones[2], ones[3], xb[j][0], xb[j][1]);
            else
              mma8<false>(isx[j], ones[0], ones[1], ones[2], ones[3], xb[j][0], xb[j][1]);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint2 bl = code_bytes<BITS>(lo[m][u]), bh = code_bytes<BITS>(hi[m][u]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              if (first)
                mma8<true>(ipart[m][j], bl.x, bh.x, bl.y, bh.y, xb[j][0], xb[j][1]);
              else
                mma8<false>(ipart[m][j], bl.x, bh.x, bl.y, bh.y, xb[j][0], xb[j][1]);
            }
          }
        }
        if (FINE || u == 3) {   // the group's (or stage's) sums, scaled
#pragma unroll
          for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = __uint_as_float(lds32(sz + (m * 16 + h * 8 + g) * 16 + sub[u]));
              if constexpr (F::INT8) {
                const int z = (int)zero_point(m, h, u);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    acc[m][j][2 * h + i] =
                        fmaf(f, (float)(ipart[m][j][2 * h + i] - z * isx[j][i]), acc[m][j][2 * h + i]);
              } else if constexpr (F::EXACT) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    acc[m][j][2 * h + i] = fmaf(f, part[m][j][2 * h + i], acc[m][j][2 * h + i]);
              } else {
                const float z = __uint_as_float(zero_point(m, h, u));   // -(B + z)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    float v = part[m][j][2 * h + i];
                    if constexpr (F::TWO) v = fmaf(1.f / (1 << BITS), odd[m][j][2 * h + i], v);
                    if constexpr (F::BASES) v = fmaf(z + 56.f, sx2[j][i], v);   // -(8 + z)
                    acc[m][j][2 * h + i] = fmaf(f, fmaf(z, sx[j][i], v), acc[m][j][2 * h + i]);
                  }
              }
            }
          }
        }
      }
      if (++slot == F::STAGES) slot = 0;
    }

    // ---- the warps' sums, then the cluster's, each in a fixed order
    constexpr int COLS = 8 * NT, CELLS = ROWS * COLS;
    const int64_t row0 = (int64_t)tile * ROWS;
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
#pragma unroll 8
        for (int w = 1; w < warps; ++w) v += red[w * CELLS + i];
        red[i] = v;                                   // cell i is this thread's alone
      }
      __syncwarp();
      cluster_sync();
    }
    for (int i = first + threadIdx.x; i < first + per; i += blockDim.x) {
      const int col = i / ROWS;
      const int64_t row = row0 + i % ROWS;
      if (col >= ntok || row >= a.p.r) continue;
      float v = 0.f;
      if (a.ctas_k > 1) {
        for (int k = 0; k < a.ctas_k; ++k) {
          float o;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(cluster_addr(red + i, k)));
          v += o;
        }
      } else {
        v = red[i];
#pragma unroll 8
        for (int w = 1; w < warps; ++w) v += red[w * CELLS + i];
      }
      if constexpr (F::INT8) v *= a.p.x_scales[tok0 + col];
      if constexpr (XT == GPTQ_F16) v *= 1.f / CODE_UNIT<BITS>;   // the codes were q times that
      if constexpr (!F::INT8)
        lost |= !(fabsf(v) <= 3.402823466e38f);
      if (a.p.bias) v += load_as_float(a.p.bias, a.p.ytype, row);
      store_float(a.p.y, a.p.ytype, (tok0 + col) * a.p.r + row, v);
    }
    if (a.ctas_k > 1) {                               // the sums stay until all have read them
      __syncwarp();
      cluster_sync();
    } else if (tile + ctas < tiles) {
      __syncthreads();                                // nor may the next tile's sums come early
    }
  }
  cp_wait<0>();
  if constexpr (!F::INT8)
    if (lost) settle_lost<BITS, NT>(a, crank, cta, ctas);
}

template <int BITS, int XT, int NT, bool FINE>
int launch_few(const PackedArgs &p, cudaStream_t st) {
  using F = Few<BITS, XT, NT, FINE>;
  constexpr size_t RED = (size_t)ROWS * 8 * NT * 4;   // a warp's sums
  static_assert(8 * (F::STAGES * F::stage_bytes(8 * NT) + F::SZWARP + RED) <= FEW_SMEM, "ring too large");
  FewArgs a{};
  a.p = p;
  a.stage_bytes = F::stage_bytes((int)(p.n < 8 * NT ? p.n : 8 * NT));
  a.aligned = (p.d / 32 * BITS) % 4 == 0 && reinterpret_cast<uintptr_t>(p.qweight) % 16 == 0;
  a.sz_aligned = (p.group < 0 ? 1 : p.d / p.group) % 4 == 0 &&
                 reinterpret_cast<uintptr_t>(p.scales) % 16 == 0 &&
                 reinterpret_cast<uintptr_t>(p.zeros) % 16 == 0;
  a.gdiv = p.group > 0 ? (uint32_t)(((1ull << 31) + p.group / 32 - 1) / (p.group / 32)) : 0;
  static std::atomic<bool> attr[64] = {};
  if (const int rc = ensure_smem_attr(packed_few_kernel<BITS, XT, NT, FINE>, FEW_SMEM, attr)) return rc;
  const int64_t tiles = (p.r + ROWS - 1) / ROWS;
  const int64_t blocks = (p.n + 8 * NT - 1) / (8 * NT);
  const int stages = (p.d + KS - 1) / KS, sms = num_sms();
  // Warps of a CTA and CTAs along k: the shape with the shortest estimate, in
  // clocks: rounds of CTAs over the tiles, each as long as its warps' stages (480
  // clocks and 110 more for each warp that shares the SM) and its sums (170 per
  // warp, 1500 more where CTAs add up theirs).  Measured, one token, 4 bits: 4096 x
  // 4096, 8 warps 5.7 us, 16 warps 6.5; 12288 x 49152, 14 warps 5 % more than 16, 8
  // warps 27 % more.
  int warps = 8, ck = 1, fit = 1;   // fit: CTAs that share an SM
  size_t smem = 0;
  int64_t best = INT64_MAX;
  for (int w = 8; w <= F::MAX_WARPS; w += 4) {
    const size_t need = (size_t)w * (F::STAGES * a.stage_bytes + F::SZWARP + RED);
    if (need > FEW_SMEM) continue;
    int res = (int)(FEW_SMEM / (need + 1024));
    if (res > 16 / w) res = 16 / w;
    if (res < 1) res = 1;
    for (int c = 1; c <= 8; c *= 2) {
      if (c > 1 && stages < w * c) break;
      const int64_t ctas = tiles * blocks * c;
      const int64_t rounds = (ctas + (int64_t)sms * res - 1) / ((int64_t)sms * res);
      const int64_t busy = ctas >= (int64_t)sms * res ? res : (ctas + sms - 1) / sms;
      const int64_t stage = 110 * w * busy + 480;
      const int64_t join = 170 * w + (c > 1 ? 1500 : 0);
      const int64_t cost = rounds * ((stages + w * c - 1) / (w * c) * stage + join) + 3000;
      if (cost <= best) best = cost, warps = w, ck = c, fit = res, smem = need;
    }
  }
  a.ctas_k = ck;
  // CTAs that fit at once walk the tiles
  int64_t clusters = (int64_t)sms * fit / (blocks * ck);
  if (clusters < 1) clusters = 1;
  if (clusters > tiles) clusters = tiles;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ck;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * ck), (unsigned)blocks);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = p.follows ? at : at + 1;
  cfg.numAttrs = (p.follows ? 1 : 0) + (ck > 1 ? 1 : 0);
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, packed_few_kernel<BITS, XT, NT, FINE>, a);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_last_error(__FILE__, __LINE__, "kernel launch", e);
    return GPTQ_ERR_CUDA;
  }
  return GPTQ_OK;
}

template <int BITS, int XT>
int launch_few_bits(const PackedArgs &p, cudaStream_t st) {
  const bool fine = p.group > 0 && p.group % KS != 0;
  if (p.n <= 8) return fine ? launch_few<BITS, XT, 1, true>(p, st) : launch_few<BITS, XT, 1, false>(p, st);
  return fine ? launch_few<BITS, XT, 2, true>(p, st) : launch_few<BITS, XT, 2, false>(p, st);
}

template <int XT>
int launch_few_type(const PackedArgs &p, cudaStream_t st) {
  switch (p.bits) {
    case 2: return launch_few_bits<2, XT>(p, st);
    case 3: return launch_few_bits<3, XT>(p, st);
    case 4: return launch_few_bits<4, XT>(p, st);
    default: return launch_few_bits<8, XT>(p, st);
  }
}

}  // namespace
}  // namespace gptq
