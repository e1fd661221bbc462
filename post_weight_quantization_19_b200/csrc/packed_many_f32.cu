// packed_many.cuh for results in fp32 (a translation unit per kind: they compile side by side).
#include "packed_many.cuh"

namespace gptq {

int launch_packed_many_f32(const PackedArgs &p, cudaStream_t st) {
  return p.xtype == GPTQ_BF16 ? launch_many_type<__nv_bfloat16, true>(p, st)
                              : launch_many_type<__half, true>(p, st);
}

}  // namespace gptq
