// What the kernels of gptq_int8_linear and gptq_int8_gated share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "activation.cuh"
#include "gptq_internal.h"

namespace gptq {

// One layer of 8-bit integers, or the two of a gated block.
struct Int8Args {
  const int8_t *x;            // [n x d]
  const float *x_scales;      // [n]
  const int8_t *w[2];         // [r x d]; gated: gate and up
  const float *w_scales[2];   // [r]
  const void *bias[2];        // [r] of ytype, or NULL
  void *y;                    // [n x r] of ytype
  int64_t n, r;
  int d, ytype, activation;
  bool gated;
  int give_up = 0;            // self-test only: GPTQ_GIVE_UP_* (gptq_selftest_int8_timeout)
};

// Self-test: whether a thread that writes results takes its wait for this tile, the last but
// one of its CTA, for run out: those of the CTA's first such warp do, or its last lane alone.
__device__ __forceinline__ bool gives_up(const Int8Args &p, int warp, int lane, int tile, int step, int tiles) {
  return (p.give_up == GPTQ_GIVE_UP_WARP || (p.give_up == GPTQ_GIVE_UP_THREAD && lane == 31)) && warp == 2 &&
         tile + step < tiles && tile + 2 * step >= tiles;
}

// How a product is launched.
struct Int8Plan {
  bool pairs;
  int ctas, cluster;          // CTAs, and of a cluster
  int tokens, rows, stages;   // per tile, rows of each layer; stages of shared memory
  int columns;                // of tensor memory, per CTA
  size_t smem;                // per CTA
};

constexpr int FEW_TOKENS = 64;
// Weights as the MMA's rows: up to FEW_TOKENS, and where int8_split is not 1; k split over
// clusters when tiles are few.  Other products: GPTQ_ERR_INVALID_ARG.
int launch_int8_single(const Int8Args &a, cudaStream_t st);
int int8_single_plan(const Int8Args &a, int sms, Int8Plan &plan);
// For more than FEW_TOKENS: the CTAs that it would split k over.
int int8_split(const Int8Args &a, int sms);
// Many tokens: pairs of CTAs, tokens as the MMA's rows.
int launch_int8_pair(const Int8Args &a, cudaStream_t st);
int int8_pair_plan(const Int8Args &a, int sms, Int8Plan &plan);
bool int8_pairs_faster(const Int8Args &a, int sms);

// A sum with its token's and row's scales, and the bias.
__device__ __forceinline__ float scaled_sum(int sum, float xs, float ws, float bias) {
  return fmaf((float)sum * xs, ws, bias);
}

// A gated result from its two sums in fp32: what a type of 16 bits takes is formed in fewer
// instructions (activate_fast).
template <int ACT, typename Y>
__device__ __forceinline__ F2 gated_pair(const F2 &g, const F2 &u) {
  if constexpr (sizeof(Y) == 2) return mul2(activate_fast<ACT, true>(g), u);
  return F2{activate<ACT>(g.x) * u.x, activate<ACT>(g.y) * u.y};
}

__device__ __forceinline__ float load_typed(const void *p, int type, int64_t i) {
  if (type == GPTQ_F16) return __half2float(reinterpret_cast<const __half *>(p)[i]);
  if (type == GPTQ_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  return reinterpret_cast<const float *>(p)[i];
}

template <typename Y>
__device__ __forceinline__ Y to_result(float v);
template <>
__device__ __forceinline__ float to_result<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half to_result<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_result<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two results of 16 bits, the first in the lower half.
template <typename Y>
__device__ __forceinline__ uint32_t to_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t to_pair<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t to_pair<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// D[tmem] (+)= A[smem] * B[smem], signed 8-bit operands, 32-bit integer sums.
__device__ __forceinline__ void umma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Boxes of a map to shared memory, by addresses: tma_load_2d, tma_load_2d_pair.
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *tmap, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const CUtensorMap *tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// A box of a map into L2.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *tmap, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y)
               : "memory");
}

// Instruction descriptor for kind::i8: 32-bit integer sums, both operands signed and K-major.
__host__ __device__ constexpr uint32_t instr_desc_i8(uint32_t M, uint32_t N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Wait for a phase, giving up where the CTA has; false then, or when the wait ran out.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, const int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (true) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*(const volatile int *)abort || global_ns() - t0 > kWaitLimitNs) return false;
  }
}

// A map of a matrix [rows x d] of 8-bit integers, loaded in boxes of box_rows rows x 128
// columns into 128-byte-swizzled shared memory; rows and columns past the end read as zeros.
int int8_map(CUtensorMap *map, const int8_t *p, int64_t rows, int d, int box_rows);

}  // namespace gptq
