// cache.cu -- the paged NVFP4 cache of keys and values: tokens quantized as they are
// written, and read back.
//
// Write: for each 16 values x of a head, with b = max |x|,
//   scale = E4M3(b / (6 alpha)),  code = E2M1(x / (scale alpha)).
// Read: code * scale * alpha.  Both move bytes: 2 or 4 per value on one side, 9/16 on
// the other.
#include <cmath>

#include "attention_device.cuh"
#include "launch_early.cuh"
#include "layer_device.cuh"

namespace nvfp4 {
namespace attention {

using layer::after_previous;
using layer::launch_early;
using bf16 = __nv_bfloat16;

constexpr int kThreads = 128;

// Row and place of one token of the call.
struct Place {
  int page;  // -1: left out
  int row;
  bool in_sequence;
};

__device__ __forceinline__ Place place_of(const CacheView& c, int t) {
  Place p = {-1, 0, false};
  const int b = find_sequence(c, t);
  Sequence s;
  if (b < 0 || !load_sequence(c, b, s) || t >= s.first + s.rows) return p;
  p.in_sequence = true;
  const int64_t j = (int64_t)s.length - s.rows + (t - s.first);
  if (j >= 0) {
    p.page = page_of(c, b, (int)j);
    p.row = (int)j % c.page_size;
  }
  if (p.page < 0) set_status(c.status, NVFP4_ERR_INDEX);
  return p;
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, bool vec, float* x) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = reinterpret_cast<const float4*>(p)[i];
        x[4 * i] = a.x;
        x[4 * i + 1] = a.y;
        x[4 * i + 2] = a.z;
        x[4 * i + 3] = a.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = layer::to_f32(p[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store16(T* p, bool vec, const float* x) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = layer::from_f32<T>(x[i]);
  }
}

// The code of x / d next to it, ties to even: the quotient is IEEE's, from the rounded
// reciprocal and the remainder (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990: exact rounding of q + r * inv for a rounded inv).
__device__ __forceinline__ float quotient(float x, float d, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, d, x), inv, q);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) write_kernel(CacheCopyArgs a, bool vec) {
  __shared__ Place at;
  const CacheView& c = a.c;
  after_previous();
  const float alpha_k = c.alpha[0], alpha_v = c.alpha[1];
  if (!(alpha_k >= 0x1p-100f && alpha_k <= 0x1p100f && alpha_v >= 0x1p-100f && alpha_v <= 0x1p100f)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(c.status, NVFP4_ERR_RANGE);
    return;
  }
  if (blockIdx.x == 0) check_batch(c);
  const int t = blockIdx.x;
  if (threadIdx.x == 0) at = place_of(c, t);
  __syncthreads();
  if (at.page < 0) return;
  const int blocks = c.dim / 16, items = c.heads * blocks * 2;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int j = i % blocks, h = i / blocks % c.heads, v = i / blocks / c.heads;
    const Tokens& src = v ? a.v : a.k;
    float x[16];
    load16(static_cast<const T*>(src.p) + (int64_t)t * src.ts + (int64_t)h * src.hs + 16 * j, vec, x);
    float b = 0.0f;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float m = fabsf(x[e]);
      if (!(m <= 3.402823466e38f)) {  // NaN or Inf
        odd = true;
        x[e] = m > 0.0f ? copysignf(3.402823466e38f, x[e]) : 0.0f;
      }
      b = fmaxf(b, fabsf(x[e]));
    }
    if (odd) set_status(c.status, NVFP4_ERR_NONFINITE);
    const float alpha = v ? alpha_v : alpha_k;
    const uint32_t s = e4m3_encode(fminf(__fdiv_rn(b, __fmul_rn(6.0f, alpha)), 1.0e6f));
    const float d = __fmul_rn(e4m3_value(s), alpha);
    const float inv = d > 0.0f ? __frcp_rn(d) : 0.0f;
    float q[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = quotient(fminf(fmaxf(x[e], -16.0f * d), 16.0f * d), d, inv);
    const int64_t co = (int64_t)at.page * c.cp + (int64_t)h * c.ch + (int64_t)at.row * c.cr;
    const int64_t so = (int64_t)at.page * c.sp + (int64_t)h * c.sh + (int64_t)at.row * c.sr;
    *reinterpret_cast<uint2*>((v ? c.vc : c.kc) + co + 8 * j) = make_uint2(e2m1x8(q), e2m1x8(q + 8));
    ((v ? c.vs : c.ks) + so)[j] = (uint8_t)s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(CacheCopyArgs a, bool vec) {
  __shared__ Place at;
  const CacheView& c = a.c;
  after_previous();
  if (blockIdx.x == 0) check_batch(c);
  const int t = blockIdx.x;
  if (threadIdx.x == 0) at = place_of(c, t);
  __syncthreads();
  if (!at.in_sequence) return;
  const float alpha_k = c.alpha[0], alpha_v = c.alpha[1];
  const int blocks = c.dim / 16, items = c.heads * blocks * 2;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int j = i % blocks, h = i / blocks % c.heads, v = i / blocks / c.heads;
    const Tokens& dst = v ? a.v : a.k;
    if (!dst.p) continue;
    float x[16] = {};
    if (at.page >= 0) {
      const int64_t co = (int64_t)at.page * c.cp + (int64_t)h * c.ch + (int64_t)at.row * c.cr;
      const int64_t so = (int64_t)at.page * c.sp + (int64_t)h * c.sh + (int64_t)at.row * c.sr;
      const uint2 w = *reinterpret_cast<const uint2*>((v ? c.vc : c.kc) + co + 8 * j);
      const float s = e4m3_value(((v ? c.vs : c.ks) + so)[j]), alpha = v ? alpha_v : alpha_k;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 p = e2m1x2_values(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xFFu);
        x[2 * e] = __fmul_rn(p.x * s, alpha);  // code * scale is exact
        x[2 * e + 1] = __fmul_rn(p.y * s, alpha);
      }
    }
    store16(static_cast<T*>(dst.p) + (int64_t)t * dst.ts + (int64_t)h * dst.hs + 16 * j, vec, x);
  }
}

// Whether all 16-value blocks of k and v begin at 16 bytes.
static bool vectors(const CacheCopyArgs& a) {
  const int64_t n = a.bf16 ? 8 : 4;
  for (const Tokens* t : {&a.k, &a.v})
    if (t->p && (reinterpret_cast<uintptr_t>(t->p) % 16 || t->ts % n || t->hs % n)) return false;
  return true;
}

}  // namespace attention

cudaError_t launch_cache_write(const CacheCopyArgs& a, cudaStream_t s) {
  using namespace attention;
  const dim3 grid((unsigned)a.c.T);
  return a.bf16 ? launch_early(write_kernel<bf16>, grid, kThreads, 0, s, a, vectors(a))
                : launch_early(write_kernel<float>, grid, kThreads, 0, s, a, vectors(a));
}
cudaError_t launch_cache_read(const CacheCopyArgs& a, cudaStream_t s) {
  using namespace attention;
  const dim3 grid((unsigned)a.c.T);
  return a.bf16 ? launch_early(read_kernel<bf16>, grid, kThreads, 0, s, a, vectors(a))
                : launch_early(read_kernel<float>, grid, kThreads, 0, s, a, vectors(a));
}

}  // namespace nvfp4
