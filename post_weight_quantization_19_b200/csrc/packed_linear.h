// What the kernels of gptq_packed_linear share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gptq_internal.h"

namespace gptq {

struct PackedArgs {
  const void *x;              // [n x d]
  const float *x_scales;      // GPTQ_I8: [n]; else NULL
  const uint32_t *qweight;    // [r x d*bits/32]
  const float *scales;        // [r x G]
  const int32_t *zeros;       // [r x G]
  const void *bias;           // [r] of ytype, or NULL
  void *y;                    // [n x r] of ytype
  int64_t n, r;
  int d, bits, group, G, xtype, ytype;
  int follows;         // x is written by a kernel just launched on the stream (griddepcontrol)
};

// Few tokens: warp-level products on codes straight from the packed rows.
int launch_packed_few_f16(const PackedArgs &a, cudaStream_t st);
int launch_packed_few_bf16(const PackedArgs &a, cudaStream_t st);
int launch_packed_few_i8(const PackedArgs &a, cudaStream_t st);
// Many tokens: weights dequantised into tensor memory, tcgen05 products.  x in
// 16 bits (xtype GPTQ_F16 or GPTQ_BF16; x_scales may still be given).
int launch_packed_many(const PackedArgs &a, cudaStream_t st);       // y in 16 bits
int launch_packed_many_f32(const PackedArgs &a, cudaStream_t st);   // y in fp32

__device__ __forceinline__ float load_as_float(const void *p, int type, int64_t i) {
  if (type == GPTQ_F16) return __half2float(reinterpret_cast<const __half *>(p)[i]);
  if (type == GPTQ_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  return reinterpret_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_float(void *p, int type, int64_t i, float v) {
  if (type == GPTQ_F16)
    reinterpret_cast<__half *>(p)[i] = __float2half_rn(v);
  else if (type == GPTQ_BF16)
    reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float *>(p)[i] = v;
}

// sum_j s (q - z) x of one row and token in 64 bits, x in 16 bits: what a result
// is where the few-token kernel's sums left the numbers -- an infinity or a NaN in x
// (it forms sum (B + q) x - (B + z) sum x, and infinities of both signs), or values
// whose multiples leave fp32 though the result does not.
template <int BITS>
__device__ __forceinline__ float sum_in_64_bits(const PackedArgs &p, int64_t tok, int64_t row) {
  const uint32_t *w = p.qweight + row * (p.d / 32) * BITS;
  double sum = 0.0;
#pragma unroll 1
  for (int j = 0; j < p.d && sum == sum; ++j) {
    const int at = j * BITS, off = at & 31;
    uint32_t q = w[at >> 5] >> off;
    if (off + BITS > 32) q |= w[(at >> 5) + 1] << (32 - off);
    const int64_t g = row * p.G + (p.group < 0 ? 0 : j / p.group);
    const int z = min(max(p.zeros[g], 0), (1 << BITS) - 1);
    sum += (double)p.scales[g] * ((int)(q & ((1u << BITS) - 1u)) - z) *
           load_as_float(p.x, p.xtype, tok * p.d + j);
  }
  return (float)sum;
}

}  // namespace gptq
