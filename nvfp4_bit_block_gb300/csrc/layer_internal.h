// layer_internal.h -- kernel launch interface of the operators around the
// linear layer, shared by libnvfp4_layer's translation units.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

struct NormArgs {
  const void* x;
  void* y;
  const void* gamma;  // nullable
  const void* beta;   // nullable
  float* mean;        // nullable
  float* rstd;        // nullable
  float* amax;        // nullable, [2]
  int64_t M, N, ldx, ldy;
  float eps;
  int x_bf16, y_bf16, w_bf16;
};

struct NormGradArgs {
  const void* dy;
  const void* x;
  const void* dres;  // nullable
  void* dx;
  const float* mean;
  const float* rstd;
  const void* gamma;  // nullable
  float* dgamma;      // nullable
  float* dbeta;       // nullable
  float* ws;
  int64_t M, N, lddy, ldx, lddres, lddx;
  int dy_bf16, x_bf16, w_bf16;
};

struct ActGradArgs {
  const void* dy;
  const void* z;  // nullable without an activation
  void* dz;       // nullable
  float* dbias;   // nullable
  float* ws;
  int64_t M, N, lddy, ldz, lddz;
  int bf16, act;
};

struct LinearArgs {
  const uint8_t* qa;
  const uint8_t* sfa;
  const float* alpha_a;
  const uint8_t* qb;
  const uint8_t* sfb;
  const float* alpha_b;
  const void* bias;      // nullable
  const void* residual;  // nullable
  void* z;               // nullable
  void* d;
  float* amax;  // nullable, [2]
  float* ws;
  int* status;  // nullable
  int64_t M, N, K, ldr, ldz, ldd;
  int bias_bf16, out_bf16, act;
};

int64_t norm_grad_workspace(int64_t M, int64_t N);
int64_t act_grad_workspace(int64_t M, int64_t N);
int64_t linear_workspace(int64_t M, int64_t N, int64_t K);

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t s);
cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s);
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);

}  // namespace nvfp4
