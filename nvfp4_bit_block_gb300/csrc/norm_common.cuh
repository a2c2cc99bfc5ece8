// norm_common.cuh -- rows held in registers: the loads, stores and reductions of
// the layer norm and its gradient.
//
// A row belongs to a group of threads, a warp or a block.  A thread holds NC
// chunks of V neighbouring values: V = 8 where rows are 16-byte aligned, 1 where
// they are not.  Chunk i of thread t is the row's chunk t + i * group, so that
// neighbouring threads touch neighbouring memory.
#pragma once

#include <atomic>

#include "layer_device.cuh"
#include "launch_early.cuh"
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
  const float zero[V] = {};
  return pack(zero, Raw<T, V>());
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

// ---- rows streamed through shared memory: a thread copies its own chunks ahead
// (cp.async) into slots that it alone reads, so that no barrier is needed and a
// group keeps several rows in flight while it works on one.
template <typename T>
__device__ __forceinline__ void copy_chunk(uint32_t dst, const T* row, int c, bool there) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16u * (uint32_t)i),
                 "l"(there ? row + c + i * (16 / (int)sizeof(T)) : row), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {  // all but the LEFT latest groups of this thread have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// The first `count` (any number) of a chunk's values, zeros after them.
template <typename T>
__device__ __forceinline__ void copy_part(uint32_t dst, const T* row, int c, int count) {
  constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const int n = min(max(count - i * kPer, 0), kPer);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16u * (uint32_t)i),
                 "l"(n > 0 ? row + c + i * kPer : row), "r"(n * (int)sizeof(T))
                 : "memory");
  }
}
// Zeros in place of the first `count` (below 8) values of a chunk that has arrived.
template <typename T>
__device__ __forceinline__ void clear_head(uint32_t at, int count) {
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    if (i < count) {
      if (sizeof(T) == 2)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 2u * i), "h"((short)0) : "memory");
      else
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4u * i), "r"(0) : "memory");
    }
  }
}
// Values lo .. hi - 1 of a chunk, the others left as they are.
template <typename T>
__device__ __forceinline__ void store_part(T* to, const Raw<T, 8>& v, int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi) to[i] = reinterpret_cast<const T*>(&v)[i];
}

// Zeros in place of a chunk's values other than lo .. hi - 1.
template <typename T>
__device__ __forceinline__ void keep_part(Raw<T, 8>& v, int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < lo || i >= hi) reinterpret_cast<T*>(&v)[i] = from_f32<T>(0.0f);
}

// 8 values as pairs for the packed fp32 instructions.
__device__ __forceinline__ void unpack2(const Raw<bf16, 8>& r, float2* f) {
  f[0] = bf16x2_to_f32x2(r.v.x);
  f[1] = bf16x2_to_f32x2(r.v.y);
  f[2] = bf16x2_to_f32x2(r.v.z);
  f[3] = bf16x2_to_f32x2(r.v.w);
}
__device__ __forceinline__ void unpack2(const Raw<float, 8>& r, float2* f) {
  f[0] = make_float2(r.v[0].x, r.v[0].y);
  f[1] = make_float2(r.v[0].z, r.v[0].w);
  f[2] = make_float2(r.v[1].x, r.v[1].y);
  f[3] = make_float2(r.v[1].z, r.v[1].w);
}
__device__ __forceinline__ Raw<bf16, 8> pack2(const float2* f, Raw<bf16, 8>) {
  Raw<bf16, 8> r;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(f[i]);
  r.v.x = *reinterpret_cast<uint32_t*>(&h[0]);
  r.v.y = *reinterpret_cast<uint32_t*>(&h[1]);
  r.v.z = *reinterpret_cast<uint32_t*>(&h[2]);
  r.v.w = *reinterpret_cast<uint32_t*>(&h[3]);
  return r;
}
__device__ __forceinline__ Raw<float, 8> pack2(const float2* f, Raw<float, 8>) {
  Raw<float, 8> r;
  r.v[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  r.v[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  return r;
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// Weights at column c as pairs, as load_weights.
__device__ __forceinline__ void load_weights2(const void* w, int is_bf16, int c, int N, float none, float2* f) {
  if (!w || c >= N) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = splat(none);
  } else if (is_bf16) {
    unpack2(*reinterpret_cast<const Raw<bf16, 8>*>(static_cast<const bf16*>(w) + c), f);
  } else {
    unpack2(*reinterpret_cast<const Raw<float, 8>*>(static_cast<const float*>(w) + c), f);
  }
}

// Largest magnitude in 8 outputs, joined to `top` (bits of the value, NaN the largest).
__device__ __forceinline__ uint32_t top_of(const Raw<bf16, 8>& r, uint32_t top) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(r.v.x), "r"(r.v.y));
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(r.v.z));
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(r.v.w));
  m &= 0x7FFF7FFFu;
  return max(top, max(m << 16, m & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t top_of(const Raw<float, 8>& r, uint32_t top) {
  float f[8];
  unpack(r, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, abs_bits(f[j]));
  return top;
}

// Sums of K values over the row's group, the same bits in every thread.  For a
// block, `buf` is K * 32 floats of shared memory, 16-byte aligned; calls alternate
// between two of them, so that one barrier per call is enough.  The warps' parts
// are read back four at a time and added in order.
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
  for (int k = 0; k < K; ++k) v[k] = 0.0f;
  for (int w = 0; w < warps; w += 4) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float4 p = *reinterpret_cast<const float4*>(buf + k * 32 + w);
      v[k] += p.x;
      if (w + 1 < warps) v[k] += p.y;
      if (w + 2 < warps) v[k] += p.z;
      if (w + 3 < warps) v[k] += p.w;
    }
  }
}

// Blocks of a kernel that an SM holds, asked for once per (device, threads, shared
// memory) and kept in a small table.  One kernel is launched with many amounts of
// shared memory, by several host threads at once: it is opted in to all that a block
// may have, whatever this call needs, so that no call lowers what another's launch
// relies on.
class BlocksPerSm {
 public:
  template <typename Kernel>
  cudaError_t get(Kernel kern, int threads, int smem, int& sms, int& per_sm) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // key: device (8 bits), threads / 32 (8), smem / 16 (16); value: SMs (16), blocks (16)
    const uint64_t key = (uint64_t)(dev & 255) << 24 | (uint64_t)(threads / 32) << 16 | (uint64_t)((smem + 15) / 16);
    std::atomic<uint64_t>& slot = seen_[(unsigned)(threads / 32) % kSlots];
    const uint64_t seen = slot.load(std::memory_order_relaxed);
    if (seen >> 32 == key && seen != 0) {
      sms = (int)(seen >> 16 & 0xFFFF);
      per_sm = (int)(seen & 0xFFFF);
      return cudaSuccess;
    }
    int most = 0;
    cudaFuncAttributes attr;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kern);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)attr.sharedSizeBytes);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    slot.store(key << 32 | (uint64_t)sms << 16 | (uint64_t)per_sm, std::memory_order_relaxed);
    return cudaSuccess;
  }

 private:
  static constexpr unsigned kSlots = 32;
  std::atomic<uint64_t> seen_[kSlots] = {};
};

inline bool rows16(const void* p, int64_t ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

// Weights at columns c .. c + 7 of a row that begins at column 0, where c may be
// below it; c mod 4 is the same in all threads.  fp32 weights inside the row are
// taken 16 bytes at a time (one by one 2500 x 777 took 10 us instead of 7).
__device__ __forceinline__ void load_weights_part(const void* w, int is_bf16, int c, int N, float none, float2* f) {
  float v[8];
  const int o = c & 3;
  if (w && !is_bf16 && reinterpret_cast<uintptr_t>(w) % 16 == 0 && c - o >= 0 && c - o + 12 <= N) {
    const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c - o);
    const float4 a = from[0], b = from[1], d = from[2];
    const float all[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float even = o & 2 ? all[i + 2] : all[i], odd = o & 2 ? all[i + 3] : all[i + 1];
      v[i] = o & 1 ? odd : even;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w && c + i >= 0 && c + i < N ? load_as_f32(w, c + i, is_bf16) : none;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

// ---- rows whose length or stride is no multiple of 8 values: row r begins r * ld
// mod 8 values after a boundary of 8 values, which is the same for
// every `period`-th row.  A block that works on such a class of rows alone has
// aligned vectors as any other: it counts columns from the boundary before the
// row's first value, and only the row's first and last chunk are partly its own.
struct RowClass {
  int period, j, shift;  // rows j, j + period, ..; values between the boundary and a row's first value
  int64_t rows;          // of the class
  __device__ RowClass(int period, int j, int64_t ld, int64_t M)
      : period(period), j(j), shift((int)(j * (ld & 7) & 7)), rows((M - j + period - 1) / period) {}
  // start of the class, counted from a tensor's first value; its rows are period * ld apart
  __device__ int64_t start(int64_t ld) const { return j * ld - shift; }
};

__host__ __device__ inline int row_period(int64_t ld) { return ld % 2 ? 8 : (ld % 4 ? 4 : (ld % 8 ? 2 : 1)); }

// Whether a tensor (or none) has row 0 on a boundary and its rows' shifts are those of stride ld.
inline bool rows_shift_as(const void* p, int64_t own_ld, int64_t ld) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (own_ld - ld) % 8 == 0);
}

}  // namespace norm
}  // namespace nvfp4
