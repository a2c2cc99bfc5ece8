// layernorm_backward.cu -- gradient of the layer norm.
#include "layer_device.cuh"
#include "layer_internal.h"

namespace nvfp4 {
namespace {

using namespace layer;

constexpr int kThreads = 256;

template <typename DT, typename XT>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float buf[32];
  const int64_t r = blockIdx.x;
  const DT* dy = static_cast<const DT*>(a.dy) + r * a.lddy;
  const XT* x = static_cast<const XT*>(a.x) + r * a.ldx;
  const XT* dres = a.dres ? static_cast<const XT*>(a.dres) + r * a.lddres : nullptr;
  XT* dx = static_cast<XT*>(a.dx) + r * a.lddx;
  const float mean = a.mean[r], rstd = a.rstd[r];
  float t0 = 0.0f, t1 = 0.0f;
  for (int64_t c = threadIdx.x; c < a.N; c += kThreads) {
    const float g = to_f32(dy[c]) * (a.gamma ? load_as_f32(a.gamma, c, a.w_bf16) : 1.0f);
    t0 += g;
    t1 += g * ((to_f32(x[c]) - mean) * rstd);
  }
  const float m0 = block_sum(t0, buf) / (float)a.N;
  const float m1 = block_sum(t1, buf) / (float)a.N;
  for (int64_t c = threadIdx.x; c < a.N; c += kThreads) {
    const float g = to_f32(dy[c]) * (a.gamma ? load_as_f32(a.gamma, c, a.w_bf16) : 1.0f);
    float v = rstd * (g - m0 - (to_f32(x[c]) - mean) * rstd * m1);
    if (dres) v += to_f32(dres[c]);
    dx[c] = from_f32<XT>(v);
  }
}

// dgamma and dbeta: a block of 32 columns x 8 row lanes, joined in shared memory.
template <typename DT, typename XT>
__global__ void __launch_bounds__(kThreads) norm_weight_grad_kernel(const NormGradArgs a) {
  __shared__ float s0[8][32], s1[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + tx;
  float t0 = 0.0f, t1 = 0.0f;
  if (c < a.N) {
    for (int64_t r = ty; r < a.M; r += 8) {
      const float dy = to_f32(static_cast<const DT*>(a.dy)[r * a.lddy + c]);
      t0 += dy;
      t1 += dy * ((to_f32(static_cast<const XT*>(a.x)[r * a.ldx + c]) - a.mean[r]) * a.rstd[r]);
    }
  }
  s0[ty][tx] = t0;
  s1[ty][tx] = t1;
  __syncthreads();
  if (ty == 0 && c < a.N) {
    for (int i = 1; i < 8; ++i) {
      t0 += s0[i][tx];
      t1 += s1[i][tx];
    }
    if (a.dbeta) a.dbeta[c] = t0;
    if (a.dgamma) a.dgamma[c] = t1;
  }
}

template <typename DT, typename XT>
void launch_grad(const NormGradArgs& a, cudaStream_t s) {
  // the weight's gradient first: dx may take dy's place
  if (a.dgamma || a.dbeta) norm_weight_grad_kernel<DT, XT><<<(unsigned)((a.N + 31) / 32), kThreads, 0, s>>>(a);
  norm_grad_kernel<DT, XT><<<(unsigned)a.M, kThreads, 0, s>>>(a);
}

}  // namespace

int64_t norm_grad_workspace(int64_t, int64_t) { return 0; }

cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  if (a.dy_bf16 && a.x_bf16) launch_grad<bf16, bf16>(a, s);
  if (a.dy_bf16 && !a.x_bf16) launch_grad<bf16, float>(a, s);
  if (!a.dy_bf16 && a.x_bf16) launch_grad<float, bf16>(a, s);
  if (!a.dy_bf16 && !a.x_bf16) launch_grad<float, float>(a, s);
  return cudaGetLastError();
}

}  // namespace nvfp4
