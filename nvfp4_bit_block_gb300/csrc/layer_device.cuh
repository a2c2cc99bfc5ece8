// layer_device.cuh -- device arithmetic shared by the operators around the
// linear layer: element types, activations and their derivatives, reductions.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "nvfp4_device.cuh"
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
// The hardware's base-2 exponential and reciprocal (about 2 and 1 units in the
// last place; subnormal results are 0, which is far below what is kept here).
__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
__device__ __forceinline__ float rcp(float t) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 2.0f * 0.7978845608028654f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kRsqrt2 = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;  // 1 / sqrt(2 pi)

// 1 / (1 + exp(-t)) of t = s / log2(e): the exponential overflows to Inf far below
// zero, where the quotient is the 0 that it should be.
__device__ __forceinline__ float sigmoid_log2(float s) { return rcp(1.0f + ex2(-s)); }

// 0.5 (1 + tanh u) = sigmoid(2u), so tanh GELU is z * sigmoid(2u): one exponential
// and one reciprocal, without the cancellation of 1 + tanh u.
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  return sigmoid_log2(z * fmaf(z * z, kLog2e * kGeluC * kGeluA, kLog2e * kGeluC));
}

// The Gaussian distribution function Phi and density at z, the latter without its
// 1 / sqrt(2 pi), for results that are rounded to bf16.  With x = |z| / sqrt 2,
// erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x): Abramowitz and Stegun,
// Handbook of Mathematical Functions, 7.1.26, off by 1.5e-7 at most; exp(-x^2) is the
// density that the derivative needs as well.  (The gradient of 16384 x 20480 in bf16: erff and expf 554 us, the
// fp32 form below 417, this 329.)
__device__ __forceinline__ void gauss(float z, float& cdf, float& density, bf16) {
  const float x = fabsf(z) * kRsqrt2;
  const float t = rcp(fmaf(0.3275911f, x, 1.0f));
  density = ex2(-kLog2e * x * x);
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q = 0.5f * q * t * density;
  cdf = z < 0.0f ? q : 1.0f - q;
}

// The same for fp32 results, as close to the formula as erff and expf bring them
// (relative error of the derivative for z ~ N(0, 1.5): 4.1e-8, that of the short form
// 9e-8).  About zero Phi = 1/2 + z B(z^2); from 1.25 on Phi(-|z|) = t A(t) exp(-z^2 / 2)
// with t = 1 / (1 + 0.4 |z|), which keeps its leading digits as it vanishes.  B and A are
// minimax fits made for this file (relative errors 1.0e-8 and 5.8e-8).  16384 x 20480
// in fp32: 616 us, HBM bound, as with the short form.
constexpr float kHalfLog2e = 0.5f * kLog2e;
__device__ __forceinline__ constexpr float gauss_b(int i) {
  constexpr float c[6] = {0.398942262f, -0.0664902106f, 0.00997228269f,
                          -0.00118383719f, 0.000111041125f, -6.80949188e-06f};
  return c[i];
}
__device__ __forceinline__ constexpr float gauss_a(int i) {
  constexpr float c[7] = {0.159597948f, 0.159060761f, 0.139282241f, 0.0545277186f,
                          0.107330345f, -0.188380703f, 0.0688984767f};
  return c[i];
}
// One value or, with the packed instructions, two (778 x 84 in fp32, where the arithmetic's
// latency counts: 10.1 instead of 10.8 us).
__device__ __forceinline__ float mul_of(float a, float b) { return a * b; }
__device__ __forceinline__ float2 mul_of(float2 a, float2 b) { return mul2(a, b); }
__device__ __forceinline__ float fma_of(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 fma_of(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float each(float v, float) { return v; }
__device__ __forceinline__ float2 each(float v, float2) { return make_float2(v, v); }
__device__ __forceinline__ float gauss_t(float z) { return rcp(fmaf(0.4f, fabsf(z), 1.0f)); }
__device__ __forceinline__ float2 gauss_t(float2 z) { return make_float2(gauss_t(z.x), gauss_t(z.y)); }
__device__ __forceinline__ float ex2_of(float v) { return ex2(v); }
__device__ __forceinline__ float2 ex2_of(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
__device__ __forceinline__ float gauss_part(float z, float mid, float tail) {
  return fabsf(z) < 1.25f ? mid : (z < 0.0f ? tail : 1.0f - tail);
}
__device__ __forceinline__ float2 gauss_part(float2 z, float2 mid, float2 tail) {
  return make_float2(gauss_part(z.x, mid.x, tail.x), gauss_part(z.y, mid.y, tail.y));
}
template <typename V>
__device__ __forceinline__ void gauss_long(V z, V& cdf, V& density) {
  const V w = mul_of(z, z), t = gauss_t(z);
  density = ex2_of(mul_of(w, each(-kHalfLog2e, z)));
  V b = each(gauss_b(5), z), q = each(gauss_a(6), z);
#pragma unroll
  for (int i = 4; i >= 0; --i) b = fma_of(b, w, each(gauss_b(i), z));
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fma_of(q, t, each(gauss_a(i), z));
  cdf = gauss_part(z, fma_of(z, b, each(0.5f, z)), mul_of(mul_of(q, t), density));
}
__device__ __forceinline__ void gauss(float z, float& cdf, float& density, float) { gauss_long(z, cdf, density); }
// Phi alone, in one piece: t V(t) exp(-z^2 / 2) with t = 1 / (1 + 0.35 |z|), a minimax fit as
// above (3.2e-8).  About zero t's rounding shows in Phi, but z Phi is small there:
// relative error of the value 3.7e-8, of the formula with erff 3.6e-8, of the short
// form 7.8e-8 (16384 x 5120 x 512 in fp32: 154 us, the two pieces 170, the short form 145).
constexpr float kGaussV = 0.35f;
__device__ __forceinline__ constexpr float gauss_v(int i) {
  constexpr float c[9] = {0.139621407f, 0.139861867f, 0.119832873f,
                          0.105507985f, -0.0231097825f, 0.159174085f,
                          -0.255714178f, 0.143971667f, -0.0291459244f};
  return c[i];
}
__device__ __forceinline__ float gauss_cdf(float z) {
  const float t = rcp(fmaf(kGaussV, fabsf(z), 1.0f)), e = ex2(z * z * -kHalfLog2e);
  float q = gauss_v(8);
#pragma unroll
  for (int i = 7; i >= 0; --i) q = fmaf(q, t, gauss_v(i));
  q = q * t * e;
  return z < 0.0f ? q : 1.0f - q;
}

// act at z for a result of type T, and below its derivative.
template <typename T>
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case NVFP4_ACT_GELU: {
      if constexpr (sizeof(T) == 4) return z * gauss_cdf(z);
      float p, e;
      gauss(z, p, e, T());
      return z * p;
    }
    case NVFP4_ACT_GELU_TANH: return z * gelu_tanh_gate(z);
    case NVFP4_ACT_SILU: return z * sigmoid_log2(z * kLog2e);
    default: return z;
  }
}

// v limited to [-c, c] (NaN becomes a limit: what it multiplies is NaN then).
__device__ __forceinline__ float limit(float v, float c) { return fminf(fmaxf(v, -c), c); }

// The derivative; with p = sigmoid(u(z)) that of z p is p + z p (1 - p) u'(z).
// Beyond the limits p (or the density) is 0 or 1 to fp32's precision, so that
// limiting z in the second term changes no finite result and keeps 0 * Inf out.
template <typename T>
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case NVFP4_ACT_GELU: {
      float p, e;
      gauss(z, p, e, T());
      return fmaf(limit(z, 16.0f) * kRsqrt2Pi, e, p);
    }
    case NVFP4_ACT_GELU_TANH: {
      const float p = gelu_tanh_gate(z), c = limit(z, 16.0f);
      return fmaf(c * fmaf(-p, p, p), fmaf(c * c, 3.0f * kGeluA * kGeluC, kGeluC), p);
    }
    case NVFP4_ACT_SILU: {
      const float p = sigmoid_log2(z * kLog2e);
      return fmaf(limit(z, 128.0f), fmaf(-p, p, p), p);
    }
    default: return 1.0f;
  }
}

// erf GELU's derivative of two values for fp32 results.
__device__ __forceinline__ float2 gelu_slope2(float2 z) {
  float2 p, e;
  gauss_long(z, p, e);
  return fma2(mul2(make_float2(limit(z.x, 16.0f), limit(z.y, 16.0f)), make_float2(kRsqrt2Pi, kRsqrt2Pi)), e, p);
}

// ---------------------------------------------------------------- reductions
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The magnitude of v as an ordered integer: larger magnitudes are larger, NaN the largest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace layer
}  // namespace nvfp4
