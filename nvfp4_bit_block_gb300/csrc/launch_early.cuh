// launch_early.cuh -- kernels that start their setup while the kernel before them
// ends, instead of one to three microseconds after it.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {
namespace layer {

// A launch that may begin while the kernel before it ends (programmatic dependent
// launch): its blocks call `after_previous` before they read or write memory.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel may do the same
}

// The amax pair zeroed for the kernel launched next, which joins its maxima to it.
static __global__ void zero_amax_kernel(float* amax) {
  after_previous();
  if (threadIdx.x < 2) amax[threadIdx.x] = 0.0f;
}
inline cudaError_t zero_amax(float* amax, cudaStream_t s) { return launch_early(zero_amax_kernel, dim3(1), 32, 0, s, amax); }

}  // namespace layer
}  // namespace nvfp4
