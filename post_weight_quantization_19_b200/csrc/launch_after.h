// Launches of kernels that set up while their predecessor on the stream drains.
#pragma once

#include <utility>

#include "gptq_internal.h"

namespace gptq {

// A kernel that calls pdl_wait_then_release before it touches memory that others write, in
// clusters of `cluster` CTAs, with the stream's own priority.
template <typename... KArgs, typename... Args>
int launch_after(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                 cudaStream_t st, Args &&...args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_last_error(__FILE__, __LINE__, "kernel launch", e);
    return GPTQ_ERR_CUDA;
  }
  return GPTQ_OK;
}

}  // namespace gptq
