// layer_device.cuh -- device arithmetic shared by the operators around the
// linear layer: element types, activations and their derivatives, reductions.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "nvfp4_layer.h"

namespace nvfp4 {
namespace layer {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) {
  return __float2bfloat16_rn(v);
}

// Element i of a vector whose type is known at run time only (weights, biases).
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int is_bf16) {
  return is_bf16 ? to_f32(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// ---------------------------------------------------------------- activations
// 1 / (1 + exp(-t)): the exponential overflows to +Inf for t below -88, where
// the quotient is the 0 that it should be.
__device__ __forceinline__ float sigmoid(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

constexpr float kGeluC = 0.7978845608028654f;     // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kRsqrt2 = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;  // 1 / sqrt(2 pi)

// 0.5 (1 + tanh u) = sigmoid(2u), so tanh GELU is z * sigmoid(2u): one
// exponential and one division, without the cancellation of 1 + tanh u.
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case NVFP4_ACT_GELU: return 0.5f * z * (1.0f + erff(z * kRsqrt2));
    case NVFP4_ACT_GELU_TANH: return z * sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
    case NVFP4_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

// v limited to [-c, c]; NaN stays NaN.
__device__ __forceinline__ float clamp_abs(float v, float c) { return v > c ? c : (v < -c ? -c : v); }

// The derivative; with p = sigmoid(u(z)) that of z p is p + z p (1 - p) u'(z).
// Beyond the clamps p (or the Gaussian) is 0 or 1 in fp32, so limiting z changes
// no finite result and keeps 0 * Inf out.
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case NVFP4_ACT_GELU: {
      const float c = clamp_abs(z, 16.0f);
      return 0.5f * (1.0f + erff(c * kRsqrt2)) + c * kRsqrt2Pi * __expf(-0.5f * c * c);
    }
    case NVFP4_ACT_GELU_TANH: {
      const float c = clamp_abs(z, 16.0f), c2 = c * c;
      const float p = sigmoid(2.0f * kGeluC * (c + kGeluA * c2 * c));
      return p + c * p * (1.0f - p) * (2.0f * kGeluC * (1.0f + 3.0f * kGeluA * c2));
    }
    case NVFP4_ACT_SILU: {
      const float c = clamp_abs(z, 128.0f);
      const float p = sigmoid(c);
      return p * (1.0f + c * (1.0f - p));
    }
    default: return 1.0f;
  }
}

// ---------------------------------------------------------------- reductions
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the block, the same bits in every thread; `buf` holds 32 floats and
// is free again after the call's last barrier.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  v = warp_sum(v);
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = warp_sum(lane < warps ? buf[lane] : 0.0f);
  __syncthreads();
  return v;
}

// The magnitude of v as an ordered integer: larger magnitudes are larger, NaN the largest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace layer
}  // namespace nvfp4
