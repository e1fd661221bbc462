// What the translation units of gptq_activation_int8 share.
#pragma once

#include "activation.cuh"
#include "gptq_internal.h"

namespace gptq {

struct ActivationArgs {
  const void *x, *up;   // [n x d] of the type; up may be NULL
  const int32_t *perm;
  int8_t *codes;
  float *scales;
  void *xhat;
  int64_t n;
  int d, activation;
};

int launch_activation_f16(const ActivationArgs &a, cudaStream_t st);
int launch_activation_bf16(const ActivationArgs &a, cudaStream_t st);

}  // namespace gptq
