// linear.cu -- the linear layer on two NVFP4 operands with bias, activation,
// residual, saved activation input and amax in its epilogue.
#include "layer_device.cuh"
#include "layer_internal.h"
#include "nvfp4_device.cuh"

namespace nvfp4 {
namespace {

using namespace layer;

constexpr int kTile = 64, kStep = 16;  // 64 x 64 outputs per block, one scale block of K per step

// Value of scale (r, c) of an operand whose K holds `cols` scale columns, in the tiled 128 x 4 layout.
__device__ __forceinline__ float scale_at(const uint8_t* sf, int64_t r, int64_t c, int64_t cols) {
  const int64_t tiles = (cols + 3) / 4;
  return e4m3_value(sf[((r / 128) * tiles + c / 4) * 512 + (r % 32) * 16 + ((r / 32) % 4) * 4 + c % 4]);
}

// Decode 16 values of each of 64 operand rows into shared memory: thread t
// takes four values of row t / 4.
__device__ __forceinline__ void load_tile(float (*s)[kTile + 1], const uint8_t* q, const uint8_t* sf, int64_t r0,
                                          int64_t rows, int64_t K, int64_t kb) {
  const int i = threadIdx.x >> 2, part = threadIdx.x & 3;
  const int64_t r = r0 + i;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (r < rows) {
    const float d = scale_at(sf, r, kb, K / 16);
    const uint32_t w = *reinterpret_cast<const uint16_t*>(q + r * (K / 2) + kb * 8 + part * 2);
    const float2 lo = e2m1x2_values(w & 0xFFu), hi = e2m1x2_values(w >> 8);
    v[0] = lo.x * d;
    v[1] = lo.y * d;
    v[2] = hi.x * d;
    v[3] = hi.y * d;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[part * 4 + j][i] = v[j];
}

template <typename T>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
  float acc[4][4] = {};
  for (int64_t kb = 0; kb < a.K / 16; ++kb) {
    load_tile(sa, a.qa, a.sfa, m0, a.M, a.K, kb);
    load_tile(sb, a.qb, a.sfb, n0, a.N, a.K, kb);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
    __syncthreads();
  }
  const float scale = a.alpha_a[0] * a.alpha_b[0];
  uint32_t top = 0;
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      float z = acc[i][j] * scale;
      if (a.bias) z += load_as_f32(a.bias, n, a.bias_bf16);
      if (a.z) static_cast<T*>(a.z)[m * a.ldz + n] = from_f32<T>(z);
      float d = act_value(z, a.act);
      if (a.residual) d += to_f32(static_cast<const T*>(a.residual)[m * a.ldr + n]);
      const T o = from_f32<T>(d);
      static_cast<T*>(a.d)[m * a.ldd + n] = o;
      top = max(top, abs_bits(to_f32(o)));
    }
  }
  if (a.amax) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) {
      atomicMax(reinterpret_cast<uint32_t*>(a.amax), top);
      atomicMax(reinterpret_cast<uint32_t*>(a.amax) + 1, top);
    }
  }
}

}  // namespace

int64_t linear_workspace(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  if (a.amax) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, 2 * sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  const int64_t gy = (a.M + kTile - 1) / kTile;
  if (gy > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)((a.N + kTile - 1) / kTile), (unsigned)gy);
  if (a.out_bf16)
    linear_kernel<bf16><<<grid, 256, 0, s>>>(a);
  else
    linear_kernel<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace nvfp4
