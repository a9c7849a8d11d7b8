// Launch of a kernel that may start while the one before it in the stream
// still runs (programmatic dependent launch).  Such a kernel calls
// griddep_wait() in every block before it touches what the earlier one writes,
// and the earlier one calls griddep_launch_dependents() when it starts.
#pragma once

#include <cuda_runtime.h>

namespace ia {

// Leave for `bytes` of dynamic shared memory.  Every kernel may use 48 KB, the
// static part (16 KB at most here) included.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  if (bytes <= 32 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool overlap, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace ia
