// layernorm.cu -- layer norm over the rows of a matrix.
//
// y = (x - mean) * rstd * gamma + beta: 2 reads and writes per element and nine
// operations, so HBM bounds it.  A row is read once and stays in registers; the
// mean is summed first and the squares about it second (two reductions: no
// cancellation however far the mean is from zero).
#include <atomic>
#include <cfloat>

#include "layer_internal.h"
#include "norm_common.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace norm {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWarpThreads = 256;  // block of the one-warp-per-row kernels

// sum / N from the sum and the rounded 1 / N, refined by the remainder sum - N * mean,
// which a fused multiply-add forms without rounding.  Of a row without spread, whose
// sum is often exact, this is the row's value; sum * (1 / N) alone may be a unit off,
// which rstd makes a visible y (-16320 in 408 columns: 0.3).  A division instead of the
// refinement took 53.5 us for 16384 x 5120 bf16, this takes 53.0 to 53.3.
__device__ __forceinline__ float mean_of(float sum, float n, float inv) {
  const float mean = sum * inv, more = fmaf(fmaf(-n, mean, sum), inv, mean);
  return fabsf(mean) <= FLT_MAX ? more : mean;  // Inf stays (its remainder is NaN)
}

// The block's largest magnitude into both amax entries: by one block alone
// stored, by several joined (the pair is zeroed before the launch).
__device__ __forceinline__ void put_amax(const NormArgs& a, uint32_t top, uint32_t* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) buf[warp] = top;
  __syncthreads();
  if (warp == 0) {
    top = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? buf[lane] : 0u);
    if (lane < 2) {
      uint32_t* p = reinterpret_cast<uint32_t*>(a.amax) + lane;
      if (gridDim.x == 1)
        *p = top;
      else
        atomicMax(p, top);
    }
  }
}

// R rows at a time per group, so that R rows share the loads of gamma and beta and
// the barriers of the reductions.
template <typename XT, typename YT, int V, int NC, int R, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a) {
  after_previous();
  __shared__ __align__(16) float buf[2][R * 32];
  __shared__ uint32_t top_s[32];
  const int N = (int)a.N;
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, group = WARP ? 32 : blockDim.x;
  const int64_t groups = WARP ? (int64_t)gridDim.x * (kWarpThreads / 32) : gridDim.x;
  const int64_t first = WARP ? (int64_t)blockIdx.x * (kWarpThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const float inv = 1.0f / (float)N;
  uint32_t top = 0;
  for (int64_t r0 = first * R; r0 < a.M; r0 += groups * R) {
    Raw<XT, V> x[R][NC];
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int i = 0; i < NC; ++i)
        x[q][i] = load_chunk<XT, V>(static_cast<const XT*>(a.x) + (r0 + q) * a.ldx, V * (lane + i * group),
                                    r0 + q < a.M ? N : 0);
    float mean[R], t[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mean[q] = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float f[V];
        unpack(x[q][i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) mean[q] += f[j];
      }
    }
    group_sums<WARP, R>(mean, buf[0]);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mean[q] = mean_of(mean[q], (float)N, inv);
      t[q] = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (V * (lane + i * group) < N) {
          float f[V];
          unpack(x[q][i], f);
#pragma unroll
          for (int j = 0; j < V; ++j) t[q] += (f[j] - mean[q]) * (f[j] - mean[q]);
        }
      }
    }
    group_sums<WARP, R>(t, buf[1]);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      t[q] = 1.0f / sqrtf(t[q] * inv + a.eps);
      if (lane == 0 && r0 + q < a.M) {
        if (a.mean) a.mean[r0 + q] = mean[q];
        if (a.rstd) a.rstd[r0 + q] = t[q];
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = V * (lane + i * group);
      if (c >= N) break;
      float g[V], b[V];
      load_weights<V>(a.gamma, a.w_bf16, c, N, 1.0f, g);
      load_weights<V>(a.beta, a.w_bf16, c, N, 0.0f, b);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (r0 + q >= a.M) break;
        float f[V];
        unpack(x[q][i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = (f[j] - mean[q]) * t[q] * g[j] + b[j];
        Raw<YT, V> o = pack(f, Raw<YT, V>());
        *reinterpret_cast<Raw<YT, V>*>(static_cast<YT*>(a.y) + (r0 + q) * a.ldy + c) = o;
        if (a.amax) {
          unpack(o, f);
#pragma unroll
          for (int j = 0; j < V; ++j) top = max(top, abs_bits(f[j]));
        }
      }
    }
  }
  if (a.amax) put_amax(a, top, top_s);
}

enum { kInRegisters, kInShared, kInMemory };

// The same for rows of vectors and many of them: S rows of each group on their way
// in shared memory, packed fp32 arithmetic.  gamma and beta stay in registers, in
// shared memory or, of the longest rows, where they are.  ODD: the rows begin at several
// places against the boundaries of 16 bytes, and a block takes those of one class;
// the values of the neighbouring rows in the row's first and last chunk count for
// nothing.
template <typename XT, typename YT, int NC, int S, bool WARP, int WEIGHTS, int THREADS, bool ODD>
__global__ void __launch_bounds__(THREADS) norm_stream_kernel(const NormArgs args) {
  after_previous();
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) float buf[2][32];
  __shared__ uint32_t top_s[32];
  const int period = ODD ? row_period(args.ldx) : 1;
  const RowClass own(period, ODD ? (int)(blockIdx.x % period) : 0, args.ldx, args.M);
  NormArgs moved;
  const NormArgs& a = ODD ? moved : args;
  if (ODD) {
    moved = args;
    moved.x = static_cast<const XT*>(args.x) + own.start(args.ldx);
    moved.y = static_cast<YT*>(args.y) + own.start(args.ldy);
    moved.ldx *= period;
    moved.ldy *= period;
    moved.M = own.rows;
  }
  const int skip = ODD ? own.shift : 0, N = (int)a.N + skip;  // the row is columns skip .. N - 1
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, group = WARP ? 32 : blockDim.x;
  const int64_t blocks = gridDim.x / period, block = blockIdx.x / period;  // of the class
  const int64_t groups = WARP ? blocks * (THREADS / 32) : blocks;
  const int64_t first = WARP ? block * (THREADS / 32) + (threadIdx.x >> 5) : block;
  const float inv = 1.0f / (float)a.N;
  // this thread's slots: [stage][chunk], blockDim.x apart
  Raw<XT, 8>* mine = reinterpret_cast<Raw<XT, 8>*>(ring) + threadIdx.x;
  const uint32_t mine_s = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  auto copy_row = [&](int64_t r, int stage) {
    if (r < a.M) {
      const XT* row = static_cast<const XT*>(a.x) + r * a.ldx;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = 8 * (lane + i * group);
        const uint32_t at = mine_s + (uint32_t)((stage * NC + i) * (int)blockDim.x * (int)sizeof(Raw<XT, 8>));
        if constexpr (ODD)
          copy_part<XT>(at, row, c, N - c);
        else
          copy_chunk<XT>(at, row, c, c < N);
      }
    }
    copies_commit();
  };
  constexpr bool kKeep = WEIGHTS == kInRegisters;
  float2 g[kKeep ? NC : 1][4], b[kKeep ? NC : 1][4];
  auto load_weights = [&](int c, float2* to_g, float2* to_b) {
    if (ODD) {
      load_weights_part(a.gamma, a.w_bf16, c - skip, (int)a.N, 1.0f, to_g);
      load_weights_part(a.beta, a.w_bf16, c - skip, (int)a.N, 0.0f, to_b);
    } else {
      load_weights2(a.gamma, a.w_bf16, c, N, 1.0f, to_g);
      load_weights2(a.beta, a.w_bf16, c, N, 0.0f, to_b);
    }
  };
  // in shared memory: per chunk two quads of gamma and two of beta, at the thread's own chunks
  float4* weights = reinterpret_cast<float4*>(mine - threadIdx.x + S * NC * (int)blockDim.x) + threadIdx.x;
  uint32_t top = 0;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) copy_row(first + s * groups, s);
  if constexpr (WEIGHTS != kInMemory) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (lane + i * group), at = kKeep ? i : 0;
      load_weights(c, g[at], b[at]);
      if (!kKeep && c < N) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 *pg = g[0] + 2 * h, *pb = b[0] + 2 * h;
          weights[(4 * i + h) * (int)blockDim.x] = make_float4(pg[0].x, pg[0].y, pg[1].x, pg[1].y);
          weights[(4 * i + 2 + h) * (int)blockDim.x] = make_float4(pb[0].x, pb[0].y, pb[1].x, pb[1].y);
        }
      }
    }
  }
  int stage = 0;
  for (int64_t r = first; r < a.M; r += groups) {
    copy_row(r + (S - 1) * groups, stage == 0 ? S - 1 : stage - 1);  // the slot read in the previous round
    copies_wait<S - 1>();
    if (ODD && lane == 0) clear_head<XT>(mine_s + (uint32_t)(stage * NC * (int)blockDim.x * (int)sizeof(Raw<XT, 8>)), skip);
    float2 x[NC][4];
    float2 sum = splat(0.0f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      unpack2(mine[(stage * NC + i) * (int)blockDim.x], x[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = add2(sum, x[i][j]);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
    float m[1] = {sum.x + sum.y};
    group_sums<WARP, 1>(m, buf[0]);
    const float mean = mean_of(m[0], (float)a.N, inv);
    const float2 shift = splat(-mean);
    sum = splat(0.0f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (8 * (lane + i * group) < N) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = add2(x[i][j], shift);
        if (ODD) {
          const int lo = skip - 8 * (lane + i * group), hi = N - 8 * (lane + i * group);
          if (lo > 0 || hi < 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (2 * j < lo || 2 * j >= hi) x[i][j].x = 0.0f;
              if (2 * j + 1 < lo || 2 * j + 1 >= hi) x[i][j].y = 0.0f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fma2(x[i][j], x[i][j], sum);
      }
    }
    float t[1] = {sum.x + sum.y};
    group_sums<WARP, 1>(t, buf[1]);
    const float rstd = 1.0f / sqrtf(t[0] * inv + a.eps);
    if (lane == 0) {
      if (a.mean) a.mean[r * period + own.j] = mean;
      if (a.rstd) a.rstd[r * period + own.j] = rstd;
    }
    YT* y = static_cast<YT*>(a.y) + r * a.ldy;
    const float2 scale = splat(rstd);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (lane + i * group);
      if (c >= N) break;
      if constexpr (WEIGHTS == kInMemory) load_weights(c, g[0], b[0]);
      if constexpr (WEIGHTS == kInShared) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 vg = weights[(4 * i + h) * (int)blockDim.x], vb = weights[(4 * i + 2 + h) * (int)blockDim.x];
          g[0][2 * h] = make_float2(vg.x, vg.y);
          g[0][2 * h + 1] = make_float2(vg.z, vg.w);
          b[0][2 * h] = make_float2(vb.x, vb.y);
          b[0][2 * h + 1] = make_float2(vb.z, vb.w);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = fma2(mul2(x[i][j], scale), g[kKeep ? i : 0][j], b[kKeep ? i : 0][j]);
      Raw<YT, 8> o = pack2(x[i], Raw<YT, 8>());
      if (!ODD || (skip <= c && c + 8 <= N)) {
        *reinterpret_cast<Raw<YT, 8>*>(y + c) = o;
      } else {
        store_part(y + c, o, skip - c, N - c);
        if (rstd > FLT_MAX) keep_part<YT>(o, skip - c, N - c);  // columns beside the row: 0 * Inf is no output
      }
      if (a.amax) top = top_of(o, top);
    }
  }
  if (a.amax) put_amax(a, top, top_s);
}

// Rows that are not 16-byte aligned: single values, NC of them per thread, with
// gamma and beta in registers and the next row's values on their way while this
// one is worked on.  Few threads with many values each: what it costs is
// instructions, and those per row and thread are shared.
template <typename XT, typename YT, int NC, bool WARP, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_scalar_kernel(const NormArgs a) {
  after_previous();
  __shared__ __align__(16) float buf[2][32];
  __shared__ uint32_t top_s[32];
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, group = WARP ? 32 : blockDim.x;
  const int64_t groups = WARP ? (int64_t)gridDim.x * (THREADS / 32) : gridDim.x;
  const int64_t first = WARP ? (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const int mine = ((int)a.N - lane + group - 1) / group;  // values of this thread: lane, lane + group, ..
  const float inv = 1.0f / (float)a.N;
  float g[NC], b[NC], x[NC];
  XT next[NC];  // as they come: a conversion here would wait for them
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    g[i] = a.gamma && i < mine ? load_as_f32(a.gamma, lane + i * group, a.w_bf16) : 1.0f;
    b[i] = a.beta && i < mine ? load_as_f32(a.beta, lane + i * group, a.w_bf16) : 0.0f;
    next[i] = from_f32<XT>(0.0f);
  }
  const XT* from = static_cast<const XT*>(a.x) + first * a.ldx + lane;
  YT* y = static_cast<YT*>(a.y) + first * a.ldy + lane;
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < mine) next[i] = from[i * group];
    from += groups * a.ldx;
  };
  if (first < a.M) load();
  uint32_t top = 0;
  for (int64_t r = first; r < a.M; r += groups, y += groups * a.ldy) {
    float s[1] = {0.0f}, t[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      x[i] = to_f32(next[i]);
      s[0] += x[i];
    }
    if (r + groups < a.M) load();
    group_sums<WARP, 1>(s, buf[0]);
    const float mean = mean_of(s[0], (float)a.N, inv);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      x[i] -= mean;
      if (i < mine) t[0] = fmaf(x[i], x[i], t[0]);
    }
    group_sums<WARP, 1>(t, buf[1]);
    const float rstd = 1.0f / sqrtf(t[0] * inv + a.eps);
    if (lane == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const YT o = from_f32<YT>(fmaf(x[i] * rstd, g[i], b[i]));
      if (i < mine) {
        y[i * group] = o;
        top = max(top, abs_bits(to_f32(o)));
      }
    }
  }
  if (a.amax) put_amax(a, top, top_s);
}

// Rows too long for the registers of a block: three passes over the row.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const NormArgs a) {
  after_previous();
  __shared__ __align__(16) float buf[2][32];
  __shared__ uint32_t top_s[32];
  uint32_t top = 0;
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + r * a.ldx;
    YT* y = static_cast<YT*>(a.y) + r * a.ldy;
    float s[1] = {0.0f}, t[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < a.N; c += kMaxThreads) s[0] += to_f32(x[c]);
    group_sums<false, 1>(s, buf[0]);
    const float mean = s[0] / (float)a.N;
    for (int64_t c = threadIdx.x; c < a.N; c += kMaxThreads) {
      const float d = to_f32(x[c]) - mean;
      t[0] += d * d;
    }
    group_sums<false, 1>(t, buf[1]);
    const float rstd = 1.0f / sqrtf(t[0] / (float)a.N + a.eps);
    for (int64_t c = threadIdx.x; c < a.N; c += kMaxThreads) {
      float v = (to_f32(x[c]) - mean) * rstd;
      if (a.gamma) v *= load_as_f32(a.gamma, c, a.w_bf16);
      if (a.beta) v += load_as_f32(a.beta, c, a.w_bf16);
      const YT o = from_f32<YT>(v);
      y[c] = o;
      top = max(top, abs_bits(to_f32(o)));
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
  if (a.amax) put_amax(a, top, top_s);
}

// `blocks` blocks of a kernel, or as many as the GPU holds at once (of either for
// each of `period` classes of rows); the amax pair is zeroed unless one block alone
// writes it.
template <auto KERN>
cudaError_t run(const NormArgs& a, int64_t blocks, int threads, cudaStream_t s, int smem = 0, int period = 1) {
  static BlocksPerSm cache;
  int sms = 0, per_sm = 0;
  cudaError_t e = cache.get(KERN, threads, smem, sms, per_sm);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sms * per_sm / period;
  blocks = (blocks < most ? blocks : (most > 0 ? most : 1)) * period;
  if (a.amax && blocks > 1) {
    e = zero_amax(a.amax, s);
    if (e != cudaSuccess) return e;
  }
  return launch_early(KERN, dim3((unsigned)blocks), threads, smem, s, a);
}

int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

// Many rows of vectors; cudaErrorNotSupported where they are too long.
template <typename XT, typename YT, bool ODD>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  // Four chunks of eight values per thread (five warps to a row of 5120 values, 53 us for 16384 x 5120 bf16; when it
  // took 58, two chunks took 69 us and one 100), three rows in flight; gamma and beta in registers as far as they fit (read
  // again for each row: 92 us).
  constexpr int kSlot = 8 * (int)sizeof(XT);  // bytes of a thread's chunk in flight
  const int64_t chunks = (a.N + (ODD ? 14 : 0)) / 8;
  const int period = ODD ? row_period(a.ldx) : 1;
  const int64_t rows = (a.M + period - 1) / period;
  if constexpr (!ODD) {  // classes begin at longer rows
    if (chunks <= 32)
      return run<norm_stream_kernel<XT, YT, 1, 4, true, kInRegisters, 256, false>>(a, (rows + 7) / 8, 256, s,
                                                                                   256 * 4 * kSlot);
    if (chunks <= 128)
      return run<norm_stream_kernel<XT, YT, 4, 3, true, kInRegisters, 256, false>>(a, (rows + 7) / 8, 256, s,
                                                                                   256 * 12 * kSlot);
  }
  const int t = round32((chunks + 3) / 4);
  if (chunks <= 1024)
    return run<norm_stream_kernel<XT, YT, 4, 3, false, kInRegisters, 256, ODD>>(a, rows, t, s, t * 12 * kSlot, period);
  if (chunks > 4096) return cudaErrorNotSupported;
  // bf16 rows leave space for the weights in shared memory (6000 x 9008: 45 us, from memory 54; fp32 101 and 97)
  const int smem = t * 8 * kSlot, with_weights = smem + t * 16 * 16;
  if constexpr (sizeof(XT) == 2) {
    if (with_weights <= 224 * 1024)
      return run<norm_stream_kernel<XT, YT, 4, 2, false, kInShared, 1024, ODD>>(a, rows, t, s, with_weights, period);
  }
  if (smem <= 224 * 1024)
    return run<norm_stream_kernel<XT, YT, 4, 2, false, kInMemory, 1024, ODD>>(a, rows, t, s, smem, period);
  return cudaErrorNotSupported;
}

template <typename XT, typename YT>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const bool vec = a.N % 8 == 0 && rows16(a.x, a.ldx, sizeof(XT)) && rows16(a.y, a.ldy, sizeof(YT)) &&
                   rows16(a.gamma, 0, 4) && rows16(a.beta, 0, 4);
  const int64_t chunks = vec ? a.N / 8 : a.N;
  const int64_t per_warp_block = kWarpThreads / 32;
  // by classes of rows where that beats single values (16384 x 2731 bf16 41 us against 49, fp32 73 and 61; 16384 x 333
  // bf16 17 and 12; 1010 x 12379 bf16 21 and 39, fp32 32 and 47)
  const bool classes = a.N > (sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 * 192 : 24 * 512) &&
                       rows_shift_as(a.x, a.ldx, a.ldx) && rows_shift_as(a.y, a.ldy, a.ldx);
  if (a.M > 608 && (vec || classes)) {
    const cudaError_t e = vec ? launch_rows<XT, YT, false>(a, s) : launch_rows<XT, YT, true>(a, s);
    if (e != cudaErrorNotSupported) return e;
  }
  if (vec) {
    if (chunks <= 128) {  // a warp holds the row
      const int64_t blocks = (a.M + 2 * per_warp_block - 1) / (2 * per_warp_block);
      return chunks <= 32 ? run<norm_kernel<XT, YT, 8, 1, 2, true, kWarpThreads>>(a, blocks, kWarpThreads, s)
                          : run<norm_kernel<XT, YT, 8, 4, 2, true, kWarpThreads>>(a, blocks, kWarpThreads, s);
    }
    if (chunks <= 1024 && a.M <= 608)  // few rows: all the threads that a row can use
      return run<norm_kernel<XT, YT, 8, 1, 1, false, 1024>>(a, a.M, round32(chunks), s);
    if (chunks <= 2048)
      return run<norm_kernel<XT, YT, 8, 4, 2, false, 512>>(a, (a.M + 1) / 2, round32((chunks + 3) / 4), s);
    if (chunks <= 4096) return run<norm_kernel<XT, YT, 8, 4, 1, false, 1024>>(a, a.M, round32((chunks + 3) / 4), s);
  } else {
    if (chunks <= 512)
      return run<norm_scalar_kernel<XT, YT, 16, true, kWarpThreads, 3>>(
          a, (a.M + per_warp_block - 1) / per_warp_block, kWarpThreads, s);
    if (chunks <= 16 * 128)
      return run<norm_scalar_kernel<XT, YT, 16, false, 128, 5>>(a, a.M, round32((chunks + 15) / 16), s);
    if (chunks <= 24 * 128)
      return run<norm_scalar_kernel<XT, YT, 24, false, 128, 4>>(a, a.M, round32((chunks + 23) / 24), s);
    if (chunks <= 24 * 256)
      return run<norm_scalar_kernel<XT, YT, 24, false, 256, 2>>(a, a.M, round32((chunks + 23) / 24), s);
    if (chunks <= 24 * 512)
      return run<norm_scalar_kernel<XT, YT, 24, false, 512, 1>>(a, a.M, round32((chunks + 23) / 24), s);
    if (chunks <= 32768) return run<norm_kernel<XT, YT, 1, 32, 1, false, 1024>>(a, a.M, round32((chunks + 31) / 32), s);
  }
  return run<norm_long_kernel<XT, YT>>(a, a.M, kMaxThreads, s);
}

}  // namespace
}  // namespace norm

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  if (a.x_bf16) return a.y_bf16 ? norm::launch<layer::bf16, layer::bf16>(a, s) : norm::launch<layer::bf16, float>(a, s);
  return a.y_bf16 ? norm::launch<float, layer::bf16>(a, s) : norm::launch<float, float>(a, s);
}

}  // namespace nvfp4
