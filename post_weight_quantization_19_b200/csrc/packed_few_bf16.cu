// packed_few.cuh for bf16 activations (a translation unit per type: they compile side by side).
#include "packed_few.cuh"

namespace gptq {

int launch_packed_few_bf16(const PackedArgs &p, cudaStream_t st) { return launch_few_type<GPTQ_BF16>(p, st); }

}  // namespace gptq
