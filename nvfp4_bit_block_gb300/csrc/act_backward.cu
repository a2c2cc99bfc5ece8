// act_backward.cu -- gradient of the linear layer's epilogue: dz = dy * act'(z)
// and the bias gradient, the column sums of dz.
#include "layer_device.cuh"
#include "layer_internal.h"

namespace nvfp4 {
namespace {

using namespace layer;

// A block of 32 columns x 8 row lanes, joined in shared memory.
template <typename T>
__global__ void __launch_bounds__(256) act_grad_kernel(const ActGradArgs a) {
  __shared__ float s0[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + tx;
  float t = 0.0f;
  if (c < a.N) {
    for (int64_t r = ty; r < a.M; r += 8) {
      const float d = to_f32(static_cast<const T*>(a.dy)[r * a.lddy + c]);
      // a product of its own (no fused add), so that dbias is the same with and without dz
      const float v = a.act ? __fmul_rn(d, act_slope(to_f32(static_cast<const T*>(a.z)[r * a.ldz + c]), a.act)) : d;
      if (a.dz) static_cast<T*>(a.dz)[r * a.lddz + c] = from_f32<T>(v);
      t += v;
    }
  }
  s0[ty][tx] = t;
  __syncthreads();
  if (ty == 0 && c < a.N && a.dbias) {
    for (int i = 1; i < 8; ++i) t += s0[i][tx];
    a.dbias[c] = t;
  }
}

}  // namespace

int64_t act_grad_workspace(int64_t, int64_t) { return 0; }

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.N + 31) / 32);
  if (a.bf16)
    act_grad_kernel<bf16><<<grid, 256, 0, s>>>(a);
  else
    act_grad_kernel<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace nvfp4
