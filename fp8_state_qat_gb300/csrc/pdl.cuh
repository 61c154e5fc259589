// pdl.cuh -- programmatic dependent launch of a chain of kernels.
#pragma once
#include <cuda_runtime.h>

namespace gdn {

// Programmatic dependent launch: a kernel's CTAs may start, and set themselves up, while the last CTAs of
// the kernel before it still run; whatever reads or overwrites that kernel's memory comes after
// dependency_wait(), which every kernel of a chain executes in each of its CTAs, so that its own end also
// stands for the end of all before it.
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;"); }

template <class... P, class... A>
inline cudaError_t launch(bool dependent, void (*kernel)(P...), dim3 grid, int threads, uint32_t smem,
                          cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gdn
