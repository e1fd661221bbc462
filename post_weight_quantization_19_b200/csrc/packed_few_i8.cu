// packed_few.cuh for 8-bit activations (a translation unit per type: they compile side by side).
#include "packed_few.cuh"

namespace gptq {

int launch_packed_few_i8(const PackedArgs &p, cudaStream_t st) { return launch_few_type<GPTQ_I8>(p, st); }

}  // namespace gptq
