// layernorm.cu -- layer norm over the rows of a matrix and its gradient.
#include "layer_device.cuh"
#include "layer_internal.h"

namespace nvfp4 {
namespace {

using namespace layer;

constexpr int kThreads = 256;

// y = (x - mean) * rstd * gamma + beta, one block per row: the mean, then the
// squares about it (no cancellation however large the mean is), then y.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs a) {
  __shared__ float buf[32];
  const int64_t r = blockIdx.x;
  const XT* x = static_cast<const XT*>(a.x) + r * a.ldx;
  YT* y = static_cast<YT*>(a.y) + r * a.ldy;
  float t = 0.0f;
  for (int64_t c = threadIdx.x; c < a.N; c += kThreads) t += to_f32(x[c]);
  const float mean = block_sum(t, buf) / (float)a.N;
  t = 0.0f;
  for (int64_t c = threadIdx.x; c < a.N; c += kThreads) {
    const float d = to_f32(x[c]) - mean;
    t += d * d;
  }
  const float rstd = 1.0f / sqrtf(block_sum(t, buf) / (float)a.N + a.eps);
  uint32_t top = 0;
  for (int64_t c = threadIdx.x; c < a.N; c += kThreads) {
    float v = (to_f32(x[c]) - mean) * rstd;
    if (a.gamma) v *= load_as_f32(a.gamma, c, a.w_bf16);
    if (a.beta) v += load_as_f32(a.beta, c, a.w_bf16);
    const YT o = from_f32<YT>(v);
    y[c] = o;
    top = max(top, abs_bits(to_f32(o)));
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
  if (a.amax) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) {
      atomicMax(reinterpret_cast<uint32_t*>(a.amax), top);
      atomicMax(reinterpret_cast<uint32_t*>(a.amax) + 1, top);
    }
  }
}

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

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  if (a.amax) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, 2 * sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)a.M;
  if (a.x_bf16 && a.y_bf16) norm_kernel<bf16, bf16><<<grid, kThreads, 0, s>>>(a);
  if (a.x_bf16 && !a.y_bf16) norm_kernel<bf16, float><<<grid, kThreads, 0, s>>>(a);
  if (!a.x_bf16 && a.y_bf16) norm_kernel<float, bf16><<<grid, kThreads, 0, s>>>(a);
  if (!a.x_bf16 && !a.y_bf16) norm_kernel<float, float><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

int64_t norm_grad_workspace(int64_t, int64_t) { return 0; }

cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  if (a.dy_bf16 && a.x_bf16) launch_grad<bf16, bf16>(a, s);
  if (a.dy_bf16 && !a.x_bf16) launch_grad<bf16, float>(a, s);
  if (!a.dy_bf16 && a.x_bf16) launch_grad<float, bf16>(a, s);
  if (!a.dy_bf16 && !a.x_bf16) launch_grad<float, float>(a, s);
  return cudaGetLastError();
}

}  // namespace nvfp4
