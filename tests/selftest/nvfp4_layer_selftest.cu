// nvfp4_layer_selftest.cu -- test-only: nvfp4_linear's kernels built with
// NVFP4_TEST_NO_COPIES, where the stages' copies are armed and never issued, so
// that every bounded wait runs out.  Both kernels have to report
// NVFP4_ERR_PIPELINE, free their tensor memory and return.
#include "layer_internal.h"
#include "nvfp4_layer.h"

extern "C" NVFP4_API int64_t nvfp4_test_linear_no_copies_workspace(int64_t M, int64_t N, int64_t K) {
  return nvfp4::linear_workspace(M, N, K);
}

extern "C" NVFP4_API int nvfp4_test_linear_no_copies(const uint8_t* qa, const uint8_t* sfa, const float* alpha_a,
                                                     const uint8_t* qb, const uint8_t* sfb, const float* alpha_b,
                                                     int64_t M, int64_t N, int64_t K, void* residual, void* d,
                                                     void* workspace, int* status, void* stream) {
  if (!qa || !sfa || !alpha_a || !qb || !sfb || !alpha_b || !d || !status) return NVFP4_ERR_NULL;
  if (M <= 0 || N <= 0 || K <= 0 || K % 32) return NVFP4_ERR_SHAPE;
  nvfp4::LinearArgs a = {};
  a.qa = qa;
  a.sfa = sfa;
  a.alpha_a = alpha_a;
  a.qb = qb;
  a.sfb = sfb;
  a.alpha_b = alpha_b;
  a.M = M;
  a.N = N;
  a.K = K;
  a.residual = residual;
  a.ldr = N;
  a.d = d;
  a.ldd = N;
  a.out_bf16 = 1;
  a.ws = static_cast<float*>(workspace);
  a.status = status;
  return nvfp4::launch_linear(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
