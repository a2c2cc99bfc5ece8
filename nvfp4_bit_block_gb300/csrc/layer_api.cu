// layer_api.cu -- the C ABI declared in include/nvfp4_layer.h: host-side
// argument validation and dispatch.  Nothing here allocates memory or keeps
// state; every call enqueues work on the caller's stream.
#include "nvfp4_layer.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "layer_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
uintptr_t elem(int is_bf16) { return is_bf16 ? 2 : 4; }
int launch_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Sizes are bounded so that row and tile counts fit 32 bits; element offsets
// are formed in 64 bits everywhere.
bool bad_size(int64_t M, int64_t N) { return M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX; }
bool bad_ld(int64_t ld, int64_t N) { return ld < N || ld > INT64_MAX / 8 / INT32_MAX; }

int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return NVFP4_OK;
  if (!ws) return NVFP4_ERR_NULL;
  if (have < need) return NVFP4_ERR_SHAPE;
  return aligned(ws, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

int zero(void* p, int64_t bytes, cudaStream_t s) {
  return p && bytes ? launch_status(cudaMemsetAsync(p, 0, (size_t)bytes, s)) : NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_layernorm(const void* x_dev, int64_t M, int64_t N, int64_t ldx, int x_is_bf16, const void* gamma_dev,
                    const void* beta_dev, int w_is_bf16, float eps, void* y_dev, int64_t ldy, int y_is_bf16,
                    float* mean_dev, float* rstd_dev, float* amax_dev, void* stream) {
  if (bad_size(M, N) || bad_ld(ldx, N) || bad_ld(ldy, N)) return NVFP4_ERR_SHAPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return NVFP4_ERR_FLAGS;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!x_dev || !y_dev)) return NVFP4_ERR_NULL;
  if (!aligned(x_dev, elem(x_is_bf16)) || !aligned(y_dev, elem(y_is_bf16)) || !aligned(gamma_dev, elem(w_is_bf16)) ||
      !aligned(beta_dev, elem(w_is_bf16)) || !aligned(mean_dev, 4) || !aligned(rstd_dev, 4) || !aligned(amax_dev, 4))
    return NVFP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return zero(amax_dev, 2 * sizeof(float), s);
  nvfp4::NormArgs a;
  a.x = x_dev;
  a.y = y_dev;
  a.gamma = gamma_dev;
  a.beta = beta_dev;
  a.mean = mean_dev;
  a.rstd = rstd_dev;
  a.amax = amax_dev;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.ldy = ldy;
  a.eps = eps;
  a.x_bf16 = x_is_bf16 ? 1 : 0;
  a.y_bf16 = y_is_bf16 ? 1 : 0;
  a.w_bf16 = w_is_bf16 ? 1 : 0;
  return launch_status(nvfp4::launch_norm(a, s));
}

int64_t nvfp4_layernorm_backward_workspace(int64_t M, int64_t N) {
  if (bad_size(M, N)) return NVFP4_ERR_SHAPE;
  return M == 0 || N == 0 ? 0 : nvfp4::norm_grad_workspace(M, N);
}

int nvfp4_layernorm_backward(const void* dy_dev, int64_t lddy, int dy_is_bf16, const void* x_dev, int64_t ldx,
                             int x_is_bf16, int64_t M, int64_t N, const float* mean_dev, const float* rstd_dev,
                             const void* gamma_dev, int w_is_bf16, const void* dres_dev, int64_t lddres, void* dx_dev,
                             int64_t lddx, float* dgamma_dev, float* dbeta_dev, void* workspace_dev,
                             int64_t workspace_bytes, void* stream) {
  if (bad_size(M, N) || bad_ld(lddy, N) || bad_ld(ldx, N) || bad_ld(lddx, N) || (dres_dev && bad_ld(lddres, N)))
    return NVFP4_ERR_SHAPE;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!dy_dev || !x_dev || !dx_dev || !mean_dev || !rstd_dev)) return NVFP4_ERR_NULL;
  if (!aligned(dy_dev, elem(dy_is_bf16)) || !aligned(x_dev, elem(x_is_bf16)) || !aligned(dx_dev, elem(x_is_bf16)) ||
      !aligned(dres_dev, elem(x_is_bf16)) || !aligned(gamma_dev, elem(w_is_bf16)) || !aligned(mean_dev, 4) ||
      !aligned(rstd_dev, 4) || !aligned(dgamma_dev, 4) || !aligned(dbeta_dev, 4))
    return NVFP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) {
    const int st = zero(dgamma_dev, N * 4, s);
    return st ? st : zero(dbeta_dev, N * 4, s);
  }
  const int st = check_workspace(workspace_dev, workspace_bytes, nvfp4::norm_grad_workspace(M, N));
  if (st) return st;
  nvfp4::NormGradArgs a;
  a.dy = dy_dev;
  a.x = x_dev;
  a.dres = dres_dev;
  a.dx = dx_dev;
  a.mean = mean_dev;
  a.rstd = rstd_dev;
  a.gamma = gamma_dev;
  a.dgamma = dgamma_dev;
  a.dbeta = dbeta_dev;
  a.ws = static_cast<float*>(workspace_dev);
  a.M = M;
  a.N = N;
  a.lddy = lddy;
  a.ldx = ldx;
  a.lddres = lddres;
  a.lddx = lddx;
  a.dy_bf16 = dy_is_bf16 ? 1 : 0;
  a.x_bf16 = x_is_bf16 ? 1 : 0;
  a.w_bf16 = w_is_bf16 ? 1 : 0;
  return launch_status(nvfp4::launch_norm_grad(a, s));
}

int64_t nvfp4_linear_workspace(int64_t M, int64_t N, int64_t K) {
  if (bad_size(M, N) || K <= 0 || K > INT32_MAX || K % 32) return NVFP4_ERR_SHAPE;
  return M == 0 || N == 0 ? 0 : nvfp4::linear_workspace(M, N, K);
}

int nvfp4_linear(const uint8_t* qa_dev, const uint8_t* sfa_dev, const float* alpha_a_dev, const uint8_t* qb_dev,
                 const uint8_t* sfb_dev, const float* alpha_b_dev, int64_t M, int64_t N, int64_t K,
                 const void* bias_dev, int bias_is_bf16, int act, const void* residual_dev, int64_t ldr, void* z_dev,
                 int64_t ldz, void* d_dev, int64_t ldd, int out_is_bf16, float* amax_dev, void* workspace_dev,
                 int64_t workspace_bytes, int* status_dev, void* stream) {
  if (bad_size(M, N) || K <= 0 || K > INT32_MAX || K % 32 || bad_ld(ldd, N) || (residual_dev && bad_ld(ldr, N)) ||
      (z_dev && bad_ld(ldz, N)))
    return NVFP4_ERR_SHAPE;
  if (act < NVFP4_ACT_NONE || act > NVFP4_ACT_SILU) return NVFP4_ERR_FLAGS;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!qa_dev || !sfa_dev || !alpha_a_dev || !qb_dev || !sfb_dev || !alpha_b_dev || !d_dev))
    return NVFP4_ERR_NULL;
  const uintptr_t oe = elem(out_is_bf16);
  if (!aligned(qa_dev, 16) || !aligned(sfa_dev, 16) || !aligned(qb_dev, 16) || !aligned(sfb_dev, 16) ||
      !aligned(alpha_a_dev, 4) || !aligned(alpha_b_dev, 4) || !aligned(bias_dev, elem(bias_is_bf16)) ||
      !aligned(residual_dev, oe) || !aligned(z_dev, oe) || !aligned(d_dev, oe) || !aligned(amax_dev, 4) ||
      !aligned(status_dev, 4))
    return NVFP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return zero(amax_dev, 2 * sizeof(float), s);
  const int st = check_workspace(workspace_dev, workspace_bytes, nvfp4::linear_workspace(M, N, K));
  if (st) return st;
  nvfp4::LinearArgs a;
  a.qa = qa_dev;
  a.sfa = sfa_dev;
  a.alpha_a = alpha_a_dev;
  a.qb = qb_dev;
  a.sfb = sfb_dev;
  a.alpha_b = alpha_b_dev;
  a.bias = bias_dev;
  a.residual = residual_dev;
  a.z = z_dev;
  a.d = d_dev;
  a.amax = amax_dev;
  a.ws = static_cast<float*>(workspace_dev);
  a.status = status_dev;
  a.M = M;
  a.N = N;
  a.K = K;
  a.ldr = ldr;
  a.ldz = ldz;
  a.ldd = ldd;
  a.bias_bf16 = bias_is_bf16 ? 1 : 0;
  a.out_bf16 = out_is_bf16 ? 1 : 0;
  a.act = act;
  return launch_status(nvfp4::launch_linear(a, s));
}

int64_t nvfp4_act_backward_workspace(int64_t M, int64_t N) {
  if (bad_size(M, N)) return NVFP4_ERR_SHAPE;
  return M == 0 || N == 0 ? 0 : nvfp4::act_grad_workspace(M, N);
}

int nvfp4_act_backward(const void* dy_dev, int64_t lddy, const void* z_dev, int64_t ldz, int64_t M, int64_t N,
                       int is_bf16, int act, void* dz_dev, int64_t lddz, float* dbias_dev, void* workspace_dev,
                       int64_t workspace_bytes, void* stream) {
  if (bad_size(M, N) || bad_ld(lddy, N) || (z_dev && bad_ld(ldz, N)) || (dz_dev && bad_ld(lddz, N)))
    return NVFP4_ERR_SHAPE;
  if (act < NVFP4_ACT_NONE || act > NVFP4_ACT_SILU) return NVFP4_ERR_FLAGS;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!dy_dev || (!z_dev && act != NVFP4_ACT_NONE))) return NVFP4_ERR_NULL;
  const uintptr_t e = elem(is_bf16);
  if (!aligned(dy_dev, e) || !aligned(z_dev, e) || !aligned(dz_dev, e) || !aligned(dbias_dev, 4))
    return NVFP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return zero(dbias_dev, N * 4, s);
  if (!dz_dev && !dbias_dev) return NVFP4_OK;
  if (dbias_dev) {
    const int st = check_workspace(workspace_dev, workspace_bytes, nvfp4::act_grad_workspace(M, N));
    if (st) return st;
  }
  nvfp4::ActGradArgs a;
  a.dy = dy_dev;
  a.z = act == NVFP4_ACT_NONE ? dy_dev : z_dev;  // without an activation z is not used
  a.dz = dz_dev;
  a.dbias = dbias_dev;
  a.ws = static_cast<float*>(workspace_dev);
  a.M = M;
  a.N = N;
  a.lddy = lddy;
  a.ldz = act == NVFP4_ACT_NONE ? lddy : ldz;
  a.lddz = lddz;
  a.bf16 = is_bf16 ? 1 : 0;
  a.act = act;
  return launch_status(nvfp4::launch_act_grad(a, s));
}

}  // extern "C"
