// norm_common.cuh -- rows held in registers: the loads, stores and reductions of
// the layer norm and its gradient.
//
// A row belongs to a group of threads, a warp or a block.  A thread holds NC
// chunks of V neighbouring values: V = 8 where rows are 16-byte aligned, 1 where
// they are not.  Chunk i of thread t is the row's chunk t + i * group, so that
// neighbouring threads touch neighbouring memory.
#pragma once

#include "layer_device.cuh"
#include "nvfp4_device.cuh"

namespace nvfp4 {
namespace norm {

using namespace layer;

// V values as they lie in memory.
template <typename T, int V>
struct Raw {
  T v[V];
};
template <>
struct Raw<bf16, 8> {
  uint4 v;
};
template <>
struct Raw<float, 8> {
  float4 v[2];
};

__device__ __forceinline__ void unpack(const Raw<bf16, 8>& r, float* f) {
  f[0] = bf16_lo(r.v.x);
  f[1] = bf16_hi(r.v.x);
  f[2] = bf16_lo(r.v.y);
  f[3] = bf16_hi(r.v.y);
  f[4] = bf16_lo(r.v.z);
  f[5] = bf16_hi(r.v.z);
  f[6] = bf16_lo(r.v.w);
  f[7] = bf16_hi(r.v.w);
}
__device__ __forceinline__ void unpack(const Raw<float, 8>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = r.v[i].x;
    f[4 * i + 1] = r.v[i].y;
    f[4 * i + 2] = r.v[i].z;
    f[4 * i + 3] = r.v[i].w;
  }
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T, 1>& r, float* f) {
  f[0] = to_f32(r.v[0]);
}
__device__ __forceinline__ Raw<bf16, 8> pack(const float* f, Raw<bf16, 8>) {
  Raw<bf16, 8> r;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  r.v.x = *reinterpret_cast<uint32_t*>(&h[0]);
  r.v.y = *reinterpret_cast<uint32_t*>(&h[1]);
  r.v.z = *reinterpret_cast<uint32_t*>(&h[2]);
  r.v.w = *reinterpret_cast<uint32_t*>(&h[3]);
  return r;
}
__device__ __forceinline__ Raw<float, 8> pack(const float* f, Raw<float, 8>) {
  Raw<float, 8> r;
  r.v[0] = make_float4(f[0], f[1], f[2], f[3]);
  r.v[1] = make_float4(f[4], f[5], f[6], f[7]);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw<T, 1> pack(const float* f, Raw<T, 1>) {
  Raw<T, 1> r;
  r.v[0] = from_f32<T>(f[0]);
  return r;
}

// Chunk at column c of a row of N values (N a multiple of V); zeros beyond it.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_chunk(const T* row, int c, int N) {
  if (c < N) return *reinterpret_cast<const Raw<T, V>*>(row + c);
  Raw<T, V> z;
  float zero[V] = {};
  z = pack(zero, z);
  return z;
}

// V weights at column c as fp32 (`one` where there are none); 16-byte aligned when V = 8.
template <int V>
__device__ __forceinline__ void load_weights(const void* w, int is_bf16, int c, int N, float none, float* f) {
  if (!w || c >= N) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = none;
  } else if (is_bf16) {
    unpack(*reinterpret_cast<const Raw<bf16, V>*>(static_cast<const bf16*>(w) + c), f);
  } else {
    unpack(*reinterpret_cast<const Raw<float, V>*>(static_cast<const float*>(w) + c), f);
  }
}

// Sums of K values over the row's group, the same bits in every thread.  For a
// block, `buf` is K * 32 floats of shared memory; calls alternate between two
// of them, so that one barrier per call is enough.
template <bool WARP, int K>
__device__ __forceinline__ void group_sums(float (&v)[K], float* buf) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (WARP) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) buf[k * 32 + warp] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < warps ? buf[k * 32 + lane] : 0.0f);
}

inline bool rows16(const void* p, int64_t ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

}  // namespace norm
}  // namespace nvfp4
