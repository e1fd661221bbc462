// gptq_activation_int8, bfloat16.
#include "activation_int8.cuh"

namespace gptq {
int launch_activation_bf16(const ActivationArgs &a, cudaStream_t st) {
  return launch_activation<__nv_bfloat16>(a, st);
}
}  // namespace gptq
