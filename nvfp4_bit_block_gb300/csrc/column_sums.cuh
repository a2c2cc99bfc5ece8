// column_sums.cuh -- the second step of sums over rows: the blocks of a gradient
// kernel each leave one row of fp32 partial sums in the workspace, and these
// rows are added in order here, so that the result does not depend on the order
// in which the blocks ran.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {
namespace colsum {

// out[v][c] = sum over p < parts of part[(p * V + v) * N + c].  A block adds 32
// columns: 32 lanes x 32 warps, each warp every 32nd row, joined in shared memory.
// It is launched while the kernel before it still runs and waits for it here.
template <int V>
__global__ void __launch_bounds__(1024) join_kernel(const float* part, int parts, int64_t N, float* out0, float* out1) {
  __shared__ float s[V][32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + tx;
  float t[V] = {};
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (c < N) {
#pragma unroll 8
    for (int p = ty; p < parts; p += 32)
#pragma unroll
      for (int v = 0; v < V; ++v) t[v] += part[((int64_t)p * V + v) * N + c];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s[v][ty][tx] = t[v];
  __syncthreads();
  // warp w adds column w's 32 parts
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float r = s[v][tx][ty];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
    float* out = v == 0 ? out0 : out1;
    const int64_t col = (int64_t)blockIdx.x * 32 + ty;
    if (tx == 0 && out && col < N) out[col] = r;
  }
}

template <int V>
cudaError_t launch_join(const float* part, int parts, int64_t N, float* out0, float* out1, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((N + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<V>, part, parts, N, out0, out1);
}

}  // namespace colsum
}  // namespace nvfp4
