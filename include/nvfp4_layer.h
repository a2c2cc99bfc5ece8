/*
 * nvfp4_layer.h -- C ABI of the operators around the NVFP4 linear layer:
 * the layer norm that makes the quantizer's input and its gradient, the
 * linear product with its bias, activation and residual, and the gradient of
 * that epilogue.  Built for GB300 (sm_103a) into libnvfp4_layer.so; status
 * values and nvfp4_strerror are those of nvfp4.h (libnvfp4.so).
 *
 * A pre-norm feed-forward block, forward and backward, from these calls and
 * those of nvfp4.h:
 *   nvfp4_layernorm (y, amax) -> nvfp4_quantize -> nvfp4_linear (activation, z,
 *   amax) -> nvfp4_quantize -> nvfp4_linear (residual);
 *   nvfp4_act_backward (bias gradients, dz) -> nvfp4_amax, nvfp4_quantize ->
 *   nvfp4_linear or nvfp4_gemm (dgrad, wgrad) -> nvfp4_layernorm_backward.
 *
 * Conventions, as in nvfp4.h: pointers named *_dev are device pointers owned by
 * the caller; the library allocates nothing and keeps nothing between calls but
 * what its kernels' launches need on a device; several host threads may call it at
 * once; every call is asynchronous on `stream` (a cudaStream_t as void*, NULL =
 * legacy default stream); argument errors are returned at once, before anything is
 * enqueued.  Matrices are row-major with a row stride in elements (ld >= columns);
 * any stride and any base address aligned to the element is accepted, rows that
 * begin and end at 16 bytes are faster; nothing between the rows is written.  An "is_bf16" argument is 1 for bf16 elements and 0
 * for fp32.  Arithmetic is fp32; a bf16 result is rounded once, to nearest even.
 * The results do not depend on the order in which blocks run: the same call
 * on the same device gives the same bits.
 * A workspace is scratch memory (16-byte aligned, contents ignored and
 * overwritten) of at least the bytes that the matching *_workspace function
 * returns on the same device; where that is 0 it may be NULL.  It must not be
 * shared by calls that may run at the same time.  The *_workspace functions
 * return a negative status for bad sizes.  A workspace that is needed and NULL is
 * ERR_NULL, one that is too small ERR_SHAPE.
 * Outputs must not overlap inputs, except where a call says that they may.
 */
#ifndef NVFP4_LAYER_H
#define NVFP4_LAYER_H

#include <stdint.h>

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of nvfp4_linear and nvfp4_act_backward. */
typedef enum {
  NVFP4_ACT_NONE = 0,
  NVFP4_ACT_RELU = 1,      /* max(z, 0); derivative 0 at z = 0                          */
  NVFP4_ACT_GELU = 2,      /* z/2 * (1 + erf(z / sqrt 2))                               */
  NVFP4_ACT_GELU_TANH = 3, /* z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3)))         */
  NVFP4_ACT_SILU = 4       /* z / (1 + exp(-z))                                         */
} nvfp4_activation;

/*
 * nvfp4_layernorm -- y = (x - mean) * rstd * gamma + beta for each row of N values,
 * with mean = sum(x)/N and rstd = 1/sqrt(sum((x - mean)^2)/N + eps).
 *
 *   x_dev        M x N, row stride ldx
 *   gamma_dev    N weights or NULL (ones);  beta_dev  N biases or NULL (zeros);
 *                both bf16 (w_is_bf16 = 1) or both fp32
 *   eps          finite and >= 0 (ERR_FLAGS otherwise)
 *   y_dev        M x N, row stride ldy; may be x_dev itself (same type and stride)
 *   mean_dev, rstd_dev  M floats each, or NULL: what the backward pass takes
 *   amax_dev     float[2] or NULL: both set to max |y| over the rounded y, as
 *                nvfp4_amax(y) without an RHT flag gives (NaN in y gives NaN), so
 *                that nvfp4_quantize can follow without another pass over y
 * M = 0 or N = 0: nothing is written but amax (0).
 * A NaN or Inf in a row makes that row NaN and touches no other.
 * Errors: SHAPE (negative sizes, ld < N), NULL, ALIGN, FLAGS, CUDA.
 */
NVFP4_API int nvfp4_layernorm(const void* x_dev, int64_t M, int64_t N, int64_t ldx, int x_is_bf16,
                              const void* gamma_dev, const void* beta_dev, int w_is_bf16, float eps, void* y_dev,
                              int64_t ldy, int y_is_bf16, float* mean_dev, float* rstd_dev, float* amax_dev,
                              void* stream);

/*
 * nvfp4_layernorm_backward -- gradients of nvfp4_layernorm.  With
 * xhat = (x - mean) * rstd and g = dy * gamma, per row
 *   dx = rstd * (g - sum(g)/N - xhat * sum(g * xhat)/N)  [+ dres],
 * and over the rows dgamma = sum(dy * xhat), dbeta = sum(dy).
 *
 *   dy_dev    M x N (stride lddy), bf16 or fp32;  x_dev  the forward pass's input
 *   mean_dev, rstd_dev  M floats each, as the forward pass wrote them
 *   gamma_dev N weights or NULL (ones), bf16 or fp32
 *   dres_dev  M x N of x's type or NULL: the gradient that reaches x past the
 *             norm (the residual branch), added to dx
 *   dx_dev    M x N of x's type; may be dy_dev or dres_dev itself (same type
 *             and stride)
 *   dgamma_dev, dbeta_dev  N floats each or NULL; overwritten (M = 0: zeros)
 *   workspace_dev  nvfp4_layernorm_backward_workspace(M, N) bytes
 * The sums over rows are formed in a fixed order.
 * Errors: SHAPE, NULL, ALIGN, CUDA.
 */
NVFP4_API int64_t nvfp4_layernorm_backward_workspace(int64_t M, int64_t N);
NVFP4_API int nvfp4_layernorm_backward(const void* dy_dev, int64_t lddy, int dy_is_bf16, const void* x_dev,
                                       int64_t ldx, int x_is_bf16, int64_t M, int64_t N, const float* mean_dev,
                                       const float* rstd_dev, const void* gamma_dev, int w_is_bf16,
                                       const void* dres_dev, int64_t lddres, void* dx_dev, int64_t lddx,
                                       float* dgamma_dev, float* dbeta_dev, void* workspace_dev,
                                       int64_t workspace_bytes, void* stream);

/*
 * nvfp4_linear -- the linear layer on two NVFP4 operands with its epilogue:
 *   z = alpha_a * alpha_b * (A * B^T) + bias,   d = act(z) + residual.
 *
 * A (M x K: the tokens) and B (N x K: the weight's rows) are operands as for
 * nvfp4_gemm: packed codes with K contiguous, E4M3 scales per 16 values along
 * K in the tiled 128 x 4 layout (NVFP4_SF_SWIZZLED; rows padded to 128, scale
 * columns to 4; the bytes of the padding are ignored).  M and N are any sizes,
 * K a multiple of 32 (a row of codes is a multiple of 16 bytes).  The products
 * are accumulated in fp32, the epilogue is fp32, and z and d are rounded once.
 *
 *   qa_dev, sfa_dev, alpha_a_dev, qb_dev, sfb_dev, alpha_b_dev   as nvfp4_gemm
 *   bias_dev      N values (bf16 or fp32) or NULL
 *   act           nvfp4_activation
 *   residual_dev  M x N of d's type (stride ldr) or NULL; may be d_dev itself
 *                 (same stride)
 *   z_dev         M x N of d's type (stride ldz) or NULL: the activation's
 *                 input, which nvfp4_act_backward takes
 *   d_dev         M x N (stride ldd), bf16 (out_is_bf16 = 1) or fp32
 *   amax_dev      float[2] or NULL: both set to max |d| over the rounded d, as
 *                 nvfp4_amax(d) without an RHT flag gives (d bf16)
 *   workspace_dev nvfp4_linear_workspace(M, N, K) bytes
 *   status_dev    int or NULL: NVFP4_ERR_PIPELINE if a tile copy or the
 *                 tensor-core work did not complete within about a second (the
 *                 outputs are then incomplete); untouched on success
 * M = 0 or N = 0: nothing is written but amax (0).  K = 0 is an error.
 * Errors: SHAPE, NULL, ALIGN (codes and scales 16-byte), FLAGS (act), CUDA.
 */
NVFP4_API int64_t nvfp4_linear_workspace(int64_t M, int64_t N, int64_t K);
NVFP4_API int nvfp4_linear(const uint8_t* qa_dev, const uint8_t* sfa_dev, const float* alpha_a_dev,
                           const uint8_t* qb_dev, const uint8_t* sfb_dev, const float* alpha_b_dev, int64_t M,
                           int64_t N, int64_t K, const void* bias_dev, int bias_is_bf16, int act,
                           const void* residual_dev, int64_t ldr, void* z_dev, int64_t ldz, void* d_dev, int64_t ldd,
                           int out_is_bf16, float* amax_dev, void* workspace_dev, int64_t workspace_bytes,
                           int* status_dev, void* stream);

/*
 * nvfp4_act_backward -- the epilogue's gradient: dz = dy * act'(z) and the bias
 * gradient dbias = sum of the unrounded dz over the rows.
 *
 *   dy_dev    M x N (stride lddy), z_dev  the forward pass's z (stride ldz);
 *             z_dev may be NULL with NVFP4_ACT_NONE
 *   is_bf16   type of dy, z and dz
 *   dz_dev    M x N (stride lddz) or NULL (only dbias is wanted); may be dy_dev
 *             or z_dev itself (same stride)
 *   dbias_dev N floats or NULL; overwritten (M = 0: zeros)
 *   workspace_dev  nvfp4_act_backward_workspace(M, N) bytes (dbias only)
 * The sum over rows is formed in a fixed order.  (A residual's gradient is dy.)
 * Errors: SHAPE, NULL, ALIGN, FLAGS (act), CUDA.
 */
NVFP4_API int64_t nvfp4_act_backward_workspace(int64_t M, int64_t N);
NVFP4_API int nvfp4_act_backward(const void* dy_dev, int64_t lddy, const void* z_dev, int64_t ldz, int64_t M,
                                 int64_t N, int is_bf16, int act, void* dz_dev, int64_t lddz, float* dbias_dev,
                                 void* workspace_dev, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_LAYER_H */
