// act_backward.cu -- gradient of the linear layer's epilogue: dz = dy * act'(z)
// and the bias gradient, the column sums of dz.
//
// Two reads and a write per element, about 20 operations: HBM bounds it.  A
// thread owns V neighbouring columns (eight, or one where rows begin anywhere) and
// walks down a band of rows with several rows' loads in flight; its column sums
// stay in registers.  Rows of an odd length begin at eight different places against
// the boundaries of 16 bytes: a block then takes every eighth row, which all begin
// alike (16384 x 2731 bf16: 55 us; value by value 98).  Each band leaves a row of
// partial sums, which join_kernel adds in order; a single band writes the result.
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
    if (sizeof(T) == 4 && V > 1 && act == NVFP4_ACT_GELU) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 p = gelu_slope2(make_float2(v[i], v[V > 1 ? i + 1 : i]));
        v[i] = p.x;
        v[V > 1 ? i + 1 : i] = p.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_slope<T>(v[i], act);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = __fmul_rn(d[i], v[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] += d[i];
  return pack(d, Raw<T, V>());
}

// Values lo .. hi - 1 of the V at a thread's columns, of rows that are not the
// thread's own beyond them.
struct Part {
  int lo, hi;
};

// Rows r0, r0 + STEP, .. below r1 of the thread's columns, R at a time.  ODD: some of
// the columns may be a neighbouring row's: they are read and add to sums that nobody
// takes, but are not written.  `end`: the row after whose last value nothing is read.
template <typename T, int V, int R, int STEP, int ACT, bool ODD>
__device__ __forceinline__ void band(const ActGradArgs& a, int64_t r0, int64_t r1, int64_t c, float* sum, Part part,
                                     int64_t end) {
  const T* dy = static_cast<const T*>(a.dy) + c;
  const T* z = static_cast<const T*>(a.z) + c;
  T* dz = static_cast<T*>(a.dz);
  const bool partly = ODD && (part.lo > 0 || part.hi < V);
  auto load = [&](const T* p, bool last) {
    if (!ODD || !last || part.hi == V) return *reinterpret_cast<const Raw<T, V>*>(p);
    Raw<T, V> v = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < part.hi) reinterpret_cast<T*>(&v)[i] = p[i];
    return v;
  };
  for (int64_t r = r0; r < r1; r += R * STEP) {
    Raw<T, V> d[R], v[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (r + q * STEP < r1) {
        const bool last = ODD && r + q * STEP == end;
        d[q] = load(dy + (r + q * STEP) * a.lddy, last);
        if (ACT) v[q] = load(z + (r + q * STEP) * a.ldz, last);
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (r + q * STEP < r1) {
        const Raw<T, V> o = slope_chunk<T, V>(d[q], v[q], ACT, sum);
        if (dz) {
          T* to = dz + (r + q * STEP) * a.lddz + c;
          if (!partly) {
            *reinterpret_cast<Raw<T, V>*>(to) = o;
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (i >= part.lo && i < part.hi) to[i] = reinterpret_cast<const T*>(&o)[i];
          }
        }
      }
    }
  }
}

// A block of TX threads across and TY down: TX * V columns of a band of rows.
// ODD: rows of one of `period` classes, blockIdx.y = band * period + class.
template <typename T, int V, int R, int TX, int TY, bool ODD>
__global__ void __launch_bounds__(TX * TY, V == 1 ? (TY > 1 ? 768 : 1024) / (TX * TY) : 0)
    act_grad_kernel(const ActGradArgs args, int64_t rows, int period) {
  after_previous();
  __shared__ float join[TY > 1 ? TY : 1][TY > 1 ? TX * V + 1 : 1];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  int64_t c = ((int64_t)blockIdx.x * TX + tx) * V, b = blockIdx.y, end = -1;
  Part part = {0, V};
  ActGradArgs moved;
  const ActGradArgs& a = ODD ? moved : args;
  if (ODD) {
    const RowClass k(period, (int)(blockIdx.y % period), args.lddy, args.M);
    b = blockIdx.y / period;
    moved = args;
    moved.dy = static_cast<const T*>(a.dy) + k.start(a.lddy);
    moved.z = static_cast<const T*>(a.z) + k.start(a.ldz);
    if (a.dz) moved.dz = static_cast<T*>(a.dz) + k.start(a.lddz);
    moved.lddy *= period;
    moved.ldz *= period;
    moved.lddz *= period;
    moved.M = k.rows;
    moved.N += k.shift;
    if ((args.M - 1) % period == k.j) end = k.rows - 1;
    part.lo = c < k.shift ? k.shift - (int)c : 0;
    part.hi = c + V > a.N ? (int)(a.N - c) : V;
  }
  const int64_t r0 = b * rows + ty, r1 = min((b + 1) * rows, a.M);
  float sum[V] = {};
  if (c < a.N) {
    switch (a.act) {  // the choice is taken once: each activation has its own loop
      case NVFP4_ACT_RELU: band<T, V, R, TY, NVFP4_ACT_RELU, ODD>(a, r0, r1, c, sum, part, end); break;
      case NVFP4_ACT_GELU: band<T, V, R, TY, NVFP4_ACT_GELU, ODD>(a, r0, r1, c, sum, part, end); break;
      case NVFP4_ACT_GELU_TANH: band<T, V, R, TY, NVFP4_ACT_GELU_TANH, ODD>(a, r0, r1, c, sum, part, end); break;
      case NVFP4_ACT_SILU: band<T, V, R, TY, NVFP4_ACT_SILU, ODD>(a, r0, r1, c, sum, part, end); break;
      default: band<T, V, R, TY, NVFP4_ACT_NONE, ODD>(a, r0, r1, c, sum, part, end); break;
    }
  }
  if (!a.dbias) return;
  float* out = gridDim.y == 1 ? a.dbias : a.ws + (int64_t)blockIdx.y * args.N;
  if constexpr (TY == 1) {
    if (c < a.N) {
      if (ODD) out += args.N - a.N;  // from the boundary's column to the row's
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!ODD || (i >= part.lo && i < part.hi)) out[c + i] = sum[i];
    }
  } else {
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
}

// Few rows: one band of narrow blocks whose threads share the rows, so that no
// second kernel is needed (it costs about 3 us).  With more rows than this, bands
// of 128-thread blocks, about eight blocks per SM.
constexpr int64_t kFewRows8 = 512, kFewRows1 = 256;
constexpr int kWide = 128;

// Rows that a thread adds one after another in fp32, at most: a sum of n values is off by up to n roundings.
// (The join adds the bands 32 apart; beyond 2^25 rows the grid's limit makes the bands longer.)
constexpr int64_t kMostRows = 512;

// Bands of rows of each of `period` classes.
int64_t bands_of(int64_t M, int64_t N, int V, int period) {
  if (M <= (V == 8 && period == 1 ? kFewRows8 : kFewRows1)) return 1;
  const int64_t strips = (N + (period > 1 ? 7 : 0) + kWide * V - 1) / (kWide * V), of_class = (M + period - 1) / period;
  const int64_t want = std::max<int64_t>(1, 152 * 8 / strips / period);
  const int64_t once = std::max<int64_t>(1, std::min(want, (M / period + kMinRows - 1) / kMinRows));
  // more in multiples of that, so that the blocks still come in whole rounds
  return std::min(once * ((of_class + once * kMostRows - 1) / (once * kMostRows)), (int64_t)65535 / period);
}

template <typename T, int V, int R, int TX, int TY, bool ODD = false>
cudaError_t run(const ActGradArgs& a, int64_t bands, cudaStream_t s, int period = 1) {
  const int64_t of_class = (a.M + period - 1) / period, rows = (of_class + bands - 1) / bands;
  const int64_t width = a.N + (ODD ? 7 : 0);
  const dim3 grid((unsigned)((width + TX * V - 1) / (TX * V)), (unsigned)((of_class + rows - 1) / rows * period));
  const cudaError_t e = launch_early(act_grad_kernel<T, V, R, TX, TY, ODD>, grid, TX * TY, 0, s, a, rows, period);
  if (e != cudaSuccess || !a.dbias || grid.y == 1) return e;
  return colsum::launch_join<1>(a.ws, (int)grid.y, a.N, a.dbias, nullptr, s);
}

template <typename T>
cudaError_t launch_t(const ActGradArgs& a, cudaStream_t s) {
  // rows in flight per thread: more cost registers and with them blocks per SM (16384 x 20480 bf16: 306 us with
  // two, 351 with four, 325 with eight)
  constexpr int R = sizeof(T) == 2 ? 2 : 1;
  const bool vec = a.N % 8 == 0 && rows16(a.dy, a.lddy, sizeof(T)) && rows16(a.z, a.ldz, sizeof(T)) &&
                   rows16(a.dz, a.lddz, sizeof(T));
  const int period = row_period(a.lddy);
  if (vec) {
    const int64_t bands = bands_of(a.M, a.N, 8, 1);
    return bands == 1 ? run<T, 8, R, 8, 32>(a, 1, s) : run<T, 8, R, kWide, 1>(a, bands, s);
  }
  // from eight values on a chunk that begins in a row ends before the end of the next
  if (a.M > kFewRows1 && a.N >= 8 && rows_shift_as(a.dy, a.lddy, a.lddy) && rows_shift_as(a.z, a.ldz, a.lddy) &&
      rows_shift_as(a.dz, a.lddz, a.lddy))
    return run<T, 8, R, kWide, 1, true>(a, bands_of(a.M, a.N, 8, period), s, period);
  const int64_t bands = bands_of(a.M, a.N, 1, 1);
  return bands == 1 ? run<T, 1, 8, 32, 8>(a, 1, s) : run<T, 1, 8, kWide, 1>(a, bands, s);
}

}  // namespace

int64_t act_grad_workspace(int64_t M, int64_t N) {
  // one row of partial sums per band and class, whatever the alignment
  int64_t bands = std::max(bands_of(M, N, 8, 1), bands_of(M, N, 1, 1));
  for (int period = 2; period <= 8 && M > kFewRows1; period *= 2)
    bands = std::max(bands, bands_of(M, N, 8, period) * period);
  return bands > 1 ? bands * N * 4 : 0;
}

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_t<layer::bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace nvfp4
