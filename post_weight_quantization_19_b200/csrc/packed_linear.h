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
int launch_packed_many(const PackedArgs &a, cudaStream_t st);

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

}  // namespace gptq
