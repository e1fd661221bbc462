// gptq_activation_int8: the arguments, and fp16.
#include <initializer_list>

#include "activation_int8.cuh"
#include "overlap.h"

namespace gptq {
int launch_activation_f16(const ActivationArgs &a, cudaStream_t st) { return launch_activation<__half>(a, st); }
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_activation_int8(const void *x, const void *up, int dtype, int64_t n, int64_t d, int activation,
                                    const int32_t *perm, int8_t *codes, float *scales, void *xhat,
                                    gptq_stream_t stream) {
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (activation < GPTQ_ACT_NONE || activation > GPTQ_ACT_GELU) return GPTQ_ERR_INVALID_ARG;
  if (n < 0 || n > (int64_t)INT32_MAX) return GPTQ_ERR_INVALID_ARG;
  if (d <= 0 || d % 32 != 0 || d > 65536) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!x || !codes || !scales) return GPTQ_ERR_INVALID_ARG;
  for (const void *p : {x, up, (const void *)codes, (const void *)xhat})
    if (reinterpret_cast<uintptr_t>(p) % 16) return GPTQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(scales) % 4 || reinterpret_cast<uintptr_t>(perm) % 4)
    return GPTQ_ERR_INVALID_ARG;
  const size_t row16 = (size_t)n * d * 2;
  const Span in[] = {{x, row16}, {up, row16}, {perm, (size_t)d * 4}};
  const Span out[] = {{codes, (size_t)n * d}, {scales, (size_t)n * 4}, {xhat, row16}};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(out[i], out[j])) return GPTQ_ERR_INVALID_ARG;
    for (const Span &s : in)
      if (overlap(out[i], s)) return GPTQ_ERR_INVALID_ARG;
  }
  const ActivationArgs a{x, up, perm, codes, scales, xhat, n, (int)d, activation};
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == GPTQ_F16 ? launch_activation_f16(a, st) : launch_activation_bf16(a, st);
}
