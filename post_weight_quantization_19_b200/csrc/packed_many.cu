// packed_many.cuh for results in 16 bits (a translation unit per kind: they compile side by side).
#include "packed_many.cuh"

namespace gptq {

int launch_packed_many(const PackedArgs &p, cudaStream_t st) {
  return p.xtype == GPTQ_BF16 ? launch_many_type<__nv_bfloat16, false>(p, st)
                              : launch_many_type<__half, false>(p, st);
}

}  // namespace gptq
