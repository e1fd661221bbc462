// gptq_selftest_activation: the activation functions by themselves, for checks of how far off
// their values are.
#include "activation.cuh"
#include "launch_after.h"
#include "overlap.h"

namespace gptq {
namespace {

// values: activate, activate_fast of any number, activate_fast of numbers of 16 bits, [3 x n];
// values64: activate64_single.
template <int ACT>
__global__ void __launch_bounds__(256) activation_values_kernel(const float *v, int64_t n, float *values, double *values64) {
  pdl_wait_then_release();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const float x = __ldcg(v + i);
  values[i] = activate<ACT>(x);
  values[n + i] = activate_fast<ACT, true>(both(x)).x;
  values[2 * n + i] = activate_fast<ACT, false>(both(x)).y;
  values64[i] = activate64_single<ACT>((double)x);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_selftest_activation(const float *v, int64_t n, int activation, float *values, double *values64,
                                        gptq_stream_t stream) {
  if (n < 0 || n > (int64_t)INT32_MAX || activation < GPTQ_ACT_NONE || activation > GPTQ_ACT_GELU)
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!v || !values || !values64 || reinterpret_cast<uintptr_t>(v) % 4 || reinterpret_cast<uintptr_t>(values) % 4 ||
      reinterpret_cast<uintptr_t>(values64) % 8)
    return GPTQ_ERR_INVALID_ARG;
  const Span in = {v, (size_t)n * 4}, out = {values, (size_t)n * 12}, out64 = {values64, (size_t)n * 8};
  if (overlap(in, out) || overlap(in, out64) || overlap(out, out64)) return GPTQ_ERR_INVALID_ARG;
  const auto kernel = activation == GPTQ_ACT_NONE   ? activation_values_kernel<GPTQ_ACT_NONE>
                      : activation == GPTQ_ACT_RELU ? activation_values_kernel<GPTQ_ACT_RELU>
                      : activation == GPTQ_ACT_SILU ? activation_values_kernel<GPTQ_ACT_SILU>
                                                    : activation_values_kernel<GPTQ_ACT_GELU>;
  return launch_after(kernel, (unsigned)((n + 255) / 256), 256, 0, 1, (cudaStream_t)stream, v, n, values, values64);
}
