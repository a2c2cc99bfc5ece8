// act_backward.cu -- gradient of the linear layer's epilogue: dz = dy * act'(z)
// and the bias gradient, the column sums of dz.
//
// Two reads and a write per element, about 20 operations: HBM bounds it.  A
// thread owns V neighbouring columns (16 bytes where rows are aligned, else one)
// and walks down a band of rows with several rows' loads in flight; its column
// sums stay in registers.  Each band leaves a row of partial sums, which
// join_kernel adds in order; a single band writes the result itself.
#include <algorithm>

#include "column_sums.cuh"
#include "layer_internal.h"
#include "norm_common.cuh"

namespace nvfp4 {
namespace {

using namespace norm;

constexpr int64_t kMinRows = 16;  // rows of a band: fewer would cost more in partial sums than they save

// dz of V values and its sums; the product is rounded on its own (no fused add),
// so that dbias is the same with and without dz.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> slope_chunk(const Raw<T, V>& dy, const Raw<T, V>& z, int act, float* sum) {
  float d[V], v[V];
  unpack(dy, d);
  if (act) {
    unpack(z, v);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = __fmul_rn(d[i], act_slope(v[i], act));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] += d[i];
  return pack(d, Raw<T, V>());
}

// Rows r0, r0 + STEP, .. below r1 of the thread's columns, R at a time.
template <typename T, int V, int R, int STEP, int ACT>
__device__ __forceinline__ void band(const ActGradArgs& a, int64_t r0, int64_t r1, int64_t c, float* sum) {
  const T* dy = static_cast<const T*>(a.dy) + c;
  const T* z = static_cast<const T*>(a.z) + c;
  T* dz = static_cast<T*>(a.dz);
  for (int64_t r = r0; r < r1; r += R * STEP) {
    Raw<T, V> d[R], v[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (r + q * STEP < r1) {
        d[q] = *reinterpret_cast<const Raw<T, V>*>(dy + (r + q * STEP) * a.lddy);
        if (ACT) v[q] = *reinterpret_cast<const Raw<T, V>*>(z + (r + q * STEP) * a.ldz);
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (r + q * STEP < r1) {
        const Raw<T, V> o = slope_chunk<T, V>(d[q], v[q], ACT, sum);
        if (dz) *reinterpret_cast<Raw<T, V>*>(dz + (r + q * STEP) * a.lddz + c) = o;
      }
    }
  }
}

// A block of TX threads across and TY down: TX * V columns of a band of rows.
template <typename T, int V, int R, int TX, int TY>
__global__ void __launch_bounds__(TX * TY, V == 1 ? 1024 / (TX * TY) : 0) act_grad_kernel(const ActGradArgs a, int64_t rows) {
  __shared__ float join[TY > 1 ? TY : 1][TY > 1 ? TX * V + 1 : 1];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int64_t c = ((int64_t)blockIdx.x * TX + tx) * V;
  const int64_t r0 = (int64_t)blockIdx.y * rows + ty, r1 = min((int64_t)(blockIdx.y + 1) * rows, a.M);
  float sum[V] = {};
  if (c < a.N) {
    switch (a.act) {  // the choice is taken once: each activation has its own loop
      case NVFP4_ACT_RELU: band<T, V, R, TY, NVFP4_ACT_RELU>(a, r0, r1, c, sum); break;
      case NVFP4_ACT_GELU: band<T, V, R, TY, NVFP4_ACT_GELU>(a, r0, r1, c, sum); break;
      case NVFP4_ACT_GELU_TANH: band<T, V, R, TY, NVFP4_ACT_GELU_TANH>(a, r0, r1, c, sum); break;
      case NVFP4_ACT_SILU: band<T, V, R, TY, NVFP4_ACT_SILU>(a, r0, r1, c, sum); break;
      default: band<T, V, R, TY, NVFP4_ACT_NONE>(a, r0, r1, c, sum); break;
    }
  }
  if (!a.dbias) return;
  float* out = gridDim.y == 1 ? a.dbias : a.ws + (int64_t)blockIdx.y * a.N;
  if (TY == 1) {
    if (c < a.N) {
#pragma unroll
      for (int i = 0; i < V; ++i) out[c + i] = sum[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) join[ty][tx * V + i] = sum[i];
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * TX * V;
  for (int i = (int)threadIdx.x; i < TX * V && c0 + i < a.N; i += TX * TY) {
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < TY; ++q) t += join[q][i];
    out[c0 + i] = t;
  }
}

// Few rows: one band of narrow blocks whose threads share the rows, so that no
// second kernel is needed (it costs about 3 us).  With more rows than this, bands
// of 128-thread blocks, about eight blocks per SM.
constexpr int64_t kFewRows8 = 512, kFewRows1 = 256;
constexpr int kWide = 128;

int64_t bands_of(int64_t M, int64_t N, int V) {
  if (M <= (V == 8 ? kFewRows8 : kFewRows1)) return 1;
  const int64_t strips = (N + kWide * V - 1) / (kWide * V);
  const int64_t want = std::max<int64_t>(1, 152 * 8 / strips);
  return std::max<int64_t>(1, std::min(want, (M + kMinRows - 1) / kMinRows));
}

template <typename T, int V, int R, int TX, int TY>
cudaError_t run(const ActGradArgs& a, int64_t bands, cudaStream_t s) {
  const int64_t rows = (a.M + bands - 1) / bands;
  const dim3 grid((unsigned)((a.N + TX * V - 1) / (TX * V)), (unsigned)((a.M + rows - 1) / rows));
  act_grad_kernel<T, V, R, TX, TY><<<grid, TX * TY, 0, s>>>(a, rows);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dbias || grid.y == 1) return e;
  return colsum::launch_join<1>(a.ws, (int)grid.y, a.N, a.dbias, nullptr, s);
}

template <typename T>
cudaError_t launch_t(const ActGradArgs& a, cudaStream_t s) {
  const bool vec = a.N % 8 == 0 && rows16(a.dy, a.lddy, sizeof(T)) && rows16(a.z, a.ldz, sizeof(T)) &&
                   rows16(a.dz, a.lddz, sizeof(T));
  const int64_t bands = bands_of(a.M, a.N, vec ? 8 : 1);
  // rows in flight per thread: more cost registers and with them blocks per SM (16384 x 20480 bf16: 306 us with
  // two, 351 with four, 325 with eight)
  constexpr int R = sizeof(T) == 2 ? 2 : 1;
  if (vec) return bands == 1 ? run<T, 8, R, 8, 32>(a, 1, s) : run<T, 8, R, kWide, 1>(a, bands, s);
  return bands == 1 ? run<T, 1, 8, 32, 8>(a, 1, s) : run<T, 1, 8, kWide, 1>(a, bands, s);
}

}  // namespace

int64_t act_grad_workspace(int64_t M, int64_t N) {
  // one row of partial sums per band, for either width
  const int64_t bands = std::max(bands_of(M, N, 8), bands_of(M, N, 1));
  return bands > 1 ? bands * N * 4 : 0;
}

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_t<layer::bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace nvfp4
