// layernorm_backward.cu -- gradient of the layer norm.
//
// With xhat = (x - mean) * rstd and g = dy * gamma, each row needs two sums,
// m0 = sum(g) / N and m1 = sum(g * xhat) / N, before its
//   dx = rstd * (g - m0 - xhat * m1) [+ dres],
// and each column the sums of dy * xhat and dy over all rows.  Two or three reads
// and a write per element, under ten packed operations: HBM bounds it.
//
// norm_grad_kernel reads everything once: a group of threads holds a row in
// registers for its two sums, walks over rows, and keeps gamma and its columns'
// two running sums in registers all the way.  Each block leaves one row of partial
// column sums (its groups joined in shared memory), which join_kernel adds in order.
// Rows of an odd length begin at up to eight places against the boundaries of 16
// bytes: a block takes those that begin alike, so that its columns stay vectors.
// Rows too long for that take two passes: the row sums, then the columns.
#include <algorithm>

#include "column_sums.cuh"
#include "layer_internal.h"
#include "norm_common.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace norm {
namespace {

constexpr int kMaxBlocks = 608;          // blocks or bands that leave a row of partial sums each; more only for kMostRows
// Rows that a thread adds one after another in fp32, at most: a sum of n values is off by up to n roundings.  (The
// join adds the blocks' sums 32 apart; beyond 2^25 rows of over 5120 values the grid's limit makes bands longer.)
constexpr int64_t kMostRows = 512;
constexpr int64_t kRing = 220 * 1024;    // shared memory for rows on their way

// Barrier of a row's group (its threads are whole warps of one block).
__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// K sums (2, 4 or 8) over a warp at once: in each of the first exchanges a lane
// keeps half of its sums and gives away the other half, so that K sums take K - 1
// exchanges and a few more instead of 5 K.  Lane l ends with sum l / (32 / K).
template <int K>
__device__ __forceinline__ float warp_sums(float (&v)[K]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = K / 2; n > 0; n >>= 1, o >>= 1) {
    const bool high = lane & o;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float give = high ? v[k] : v[k + n], keep = high ? v[k + n] : v[k];
      v[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
  }
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
  return v[0];
}

// K sums over a group of `warps` warps, the same bits in all its threads; `buf` is
// the group's, calls alternate between two of them.
template <int K>
__device__ __forceinline__ void group_sums_k(float (&v)[K], float* buf, int warps, int group) {
  constexpr int L = 32 / K;  // lanes that share a sum
  const int lane = threadIdx.x & 31, k = lane / L, l = lane % L;
  float t = warp_sums<K>(v);
  if (warps > 1) {
    if (l == 0) buf[K * ((int)(threadIdx.x >> 5) - group * warps) + k] = t;
    group_sync(1 + group, warps * 32);
    t = 0.0f;
#pragma unroll 1
    for (int w = l; w < warps; w += L) t += buf[K * w + k];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  }
#pragma unroll
  for (int q = 0; q < K; ++q) v[q] = __shfl_sync(0xFFFFFFFFu, t, q * L);
}

// 16-byte pieces of shared memory at a 32-bit address, read anew each time.
template <typename T>
__device__ __forceinline__ Raw<T, 8> slot_read(uint32_t at) {
  Raw<T, 8> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(r) / 16; ++i) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + 16u * i));
    reinterpret_cast<uint4*>(&r)[i] = v;
  }
  return r;
}
// Chunks of a thread as pairs of neighbours.
template <typename T, int NC>
__device__ __forceinline__ void to_pairs(const Raw<T, 8> (&raw)[NC], float2 (&f)[NC * 4]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) unpack2(raw[i], f + 4 * i);
}

// R neighbouring rows at a time, which share a barrier, the sums' exchanges and the
// loop's overhead.  S times R rows of each group are in shared memory or on their
// way there; dy and x are read from it again after the sums instead of being
// kept in registers.  ODD: the rows are one of `period` classes, of class
// blockIdx.x mod period; the values of the neighbouring rows in the row's first
// and last chunk count as zeros.
template <typename DT, typename XT, int NC, int R, int S, bool RES, int THREADS, int BLOCKS, bool ODD>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    norm_grad_kernel(const NormGradArgs args, int group_threads, int row_classes) {
  after_previous();
  constexpr int P = NC * 4, K = R == 3 ? 8 : 2 * R;  // sums of a round, a power of two
  extern __shared__ uint4 ring[];
  __shared__ float buf[2][THREADS / 32 * K];
  const int period = ODD ? row_classes : 1;
  const RowClass own(period, ODD ? (int)(blockIdx.x % period) : 0, args.ldx, args.M);
  NormGradArgs moved;
  const NormGradArgs& a = ODD ? moved : args;
  if (ODD) {
    moved = args;
    moved.dy = static_cast<const DT*>(args.dy) + own.start(args.lddy);
    moved.x = static_cast<const XT*>(args.x) + own.start(args.ldx);
    if (RES) moved.dres = static_cast<const XT*>(args.dres) + own.start(args.lddres);
    moved.dx = static_cast<XT*>(args.dx) + own.start(args.lddx);
    moved.lddy *= period;
    moved.ldx *= period;
    moved.lddres *= period;
    moved.lddx *= period;
    moved.M = own.rows;
  }
  const int skip = ODD ? own.shift : 0, N = (int)a.N + skip;  // the row is columns skip .. N - 1
  const int warps = group_threads >> 5, group = (int)threadIdx.x / group_threads, ngroups = (int)blockDim.x / group_threads;
  const int t = (int)threadIdx.x - group * group_threads;
  const int64_t step = (int64_t)(gridDim.x / period) * ngroups * R;
  const int64_t first = ((int64_t)(blockIdx.x / period) * ngroups + group) * R;
  const float inv = 1.0f / (float)a.N;
  // this thread's slots: per stage and row NC chunks of dy, of x and of dres, each blockDim.x apart
  constexpr uint32_t kDy = sizeof(Raw<DT, 8>), kX = sizeof(Raw<XT, 8>);
  const uint32_t threads = blockDim.x, at_x = NC * threads * kDy, at_res = at_x + NC * threads * kX;
  const uint32_t row_bytes = at_x + NC * threads * kX * (RES ? 2 : 1), stage_bytes = R * row_bytes;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t my_dy = base + threadIdx.x * kDy, my_x = base + at_x + threadIdx.x * kX;
  // global positions: the rows being copied, the rows being worked on
  const DT* dy = static_cast<const DT*>(a.dy) + first * a.lddy + 8 * t;
  const XT* x = static_cast<const XT*>(a.x) + first * a.ldx + 8 * t;
  const XT* res = RES ? static_cast<const XT*>(a.dres) + first * a.lddres + 8 * t : nullptr;
  XT* dx = static_cast<XT*>(a.dx) + first * a.lddx + 8 * t;
  int64_t ahead = first;  // row that dy, x and res point at
  auto copy_rows = [&](uint32_t stage) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (ahead + q < a.M) {
        const uint32_t at = stage + q * row_bytes;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int off = 8 * i * group_threads;
          if constexpr (ODD) {
            const int there = N - 8 * t - off;
            copy_part<DT>(my_dy + at + i * threads * kDy, dy + q * a.lddy, off, there);
            copy_part<XT>(my_x + at + i * threads * kX, x + q * a.ldx, off, there);
            if constexpr (RES) copy_part<XT>(my_x + (at_res - at_x) + at + i * threads * kX, res + q * a.lddres, off, there);
          } else {
            const bool there = 8 * t + off < N;
            copy_chunk<DT>(my_dy + at + i * threads * kDy, dy + q * a.lddy, off, there);
            copy_chunk<XT>(my_x + at + i * threads * kX, x + q * a.ldx, off, there);
            if constexpr (RES) copy_chunk<XT>(my_x + (at_res - at_x) + at + i * threads * kX, res + q * a.lddres, off, there);
          }
        }
      }
    }
    dy += step * a.lddy;
    x += step * a.ldx;
    if constexpr (RES) res += step * a.lddres;
    ahead += step;
    copies_commit();
  };
  float2 gamma[P], dg[P], db[P];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (ODD)
      load_weights_part(a.gamma, a.w_bf16, 8 * (t + i * group_threads) - skip, (int)a.N, 1.0f, gamma + 4 * i);
    else
      load_weights2(a.gamma, a.w_bf16, 8 * (t + i * group_threads), N, 1.0f, gamma + 4 * i);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) dg[p] = db[p] = splat(0.0f);
#pragma unroll
  for (int s = 0; s < S - 1; ++s) copy_rows((uint32_t)s * stage_bytes);
  float mean[R], rstd[R];
  auto load_stats = [&](int64_t r) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mean[q] = r + q < a.M ? a.mean[(r + q) * period + own.j] : 0.0f;
      rstd[q] = r + q < a.M ? a.rstd[(r + q) * period + own.j] : 0.0f;
    }
  };
  load_stats(first);
  uint32_t stage = 0;
  int parity = 0;
  float* mine = buf[0] + group * warps * K;
  for (int64_t r = first; r < a.M; r += step, dx += step * a.lddx) {
    float2 d[R][P], xh[R][P];
    Raw<XT, 8> raw_r[NC];
    auto read = [&](int q) {  // row q's dy and x from its slots
      Raw<DT, 8> raw_d[NC];
      Raw<XT, 8> raw_x[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        raw_d[i] = slot_read<DT>(my_dy + stage + q * row_bytes + i * threads * kDy);
        raw_x[i] = slot_read<XT>(my_x + stage + q * row_bytes + i * threads * kX);
      }
      to_pairs(raw_d, d[q]);
      to_pairs(raw_x, xh[q]);
    };
    copy_rows(stage == 0 ? (S - 1) * stage_bytes : stage - stage_bytes);  // the slots read in the previous round
    copies_wait<S - 1>();
    if (ODD && t == 0) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        clear_head<DT>(my_dy + stage + q * row_bytes, skip);
        clear_head<XT>(my_x + stage + q * row_bytes, skip);
      }
    }
    float2 scale[R], shift[R];
    float sums[K];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      scale[q] = splat(rstd[q]);
      shift[q] = splat(-mean[q]);
    }
    load_stats(r + step);  // the next rows', long before they are needed
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 s0 = splat(0.0f), s1 = splat(0.0f);
      read(q);
      if (R == 1 || r + q < a.M) {  // slots of a row that is not there hold old values
#pragma unroll
        for (int p = 0; p < P; ++p) {  // beyond the row dy is 0, so that nothing is added
          xh[q][p] = mul2(add2(xh[q][p], shift[q]), scale[q]);
          db[p] = add2(db[p], d[q][p]);
          dg[p] = fma2(d[q][p], xh[q][p], dg[p]);
          d[q][p] = mul2(d[q][p], gamma[p]);
          s0 = add2(s0, d[q][p]);
          s1 = fma2(d[q][p], xh[q][p], s1);
        }
      }
      sums[2 * q] = s0.x + s0.y;
      sums[2 * q + 1] = s1.x + s1.y;
    }
#pragma unroll
    for (int k = 2 * R; k < K; ++k) sums[k] = 0.0f;
    group_sums_k<K>(sums, mine + parity * (THREADS / 32 * K), warps, group);
    parity ^= 1;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (R > 1 && r + q >= a.M) break;
      read(q);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        xh[q][p] = mul2(add2(xh[q][p], shift[q]), scale[q]);
        d[q][p] = mul2(d[q][p], gamma[p]);
      }
      const float2 k0 = splat(-sums[2 * q] * inv * scale[q].x), k1 = splat(-sums[2 * q + 1] * inv);
#pragma unroll
      for (int p = 0; p < P; ++p) d[q][p] = fma2(fma2(xh[q][p], k1, d[q][p]), scale[q], k0);
      if constexpr (RES) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          raw_r[i] = slot_read<XT>(my_x + (at_res - at_x) + stage + q * row_bytes + i * threads * kX);
        to_pairs(raw_r, xh[q]);
#pragma unroll
        for (int p = 0; p < P; ++p) d[q][p] = add2(d[q][p], xh[q][p]);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int off = 8 * i * group_threads;
        if (8 * t + off < N) {
          XT* o = dx + q * a.lddx + off;
          const Raw<XT, 8> v = pack2(d[q] + 4 * i, Raw<XT, 8>());
          const int lo = skip - 8 * t - off, hi = N - 8 * t - off;
          if (!ODD || (lo <= 0 && hi >= 8))
            *reinterpret_cast<Raw<XT, 8>*>(o) = v;
          else
            store_part(o, v, lo, hi);
        }
      }
    }
    stage = stage == (S - 1) * stage_bytes ? 0 : stage + stage_bytes;
  }
  if (!a.dgamma && !a.dbeta) return;
  // one row of column sums per block; alone it is the result
  float* out_g = gridDim.x == 1 ? a.dgamma : a.ws + (int64_t)blockIdx.x * 2 * a.N;
  float* out_b = gridDim.x == 1 ? a.dbeta : a.ws + ((int64_t)blockIdx.x * 2 + 1) * a.N;
  // the groups' sums side by side in shared memory, then added in order, a column per thread
  float* sums = reinterpret_cast<float*>(ring);  // [group][2][width]
  const int width = group_threads * NC * 8;
  copies_wait<0>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float4* to = reinterpret_cast<float4*>(sums + group * 2 * width + 8 * (t + i * group_threads));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = 4 * i + 2 * h;
      to[h] = make_float4(dg[p].x, dg[p].y, dg[p + 1].x, dg[p + 1].y);
      to[h + width / 4] = make_float4(db[p].x, db[p].y, db[p + 1].x, db[p + 1].y);
    }
  }
  __syncthreads();
  for (int c = (int)threadIdx.x; c < (int)a.N; c += (int)blockDim.x) {
    float vg = 0.0f, vb = 0.0f;
    for (int q = 0; q < ngroups; ++q) {
      vg += sums[q * 2 * width + skip + c];
      vb += sums[q * 2 * width + width + skip + c];
    }
    if (out_g) out_g[c] = vg;
    if (out_b) out_b[c] = vb;
  }
}

// Rows that are not 16-byte aligned: single values, NC of them per thread, the next
// row's on their way (unconverted: a conversion would wait for them) while this
// one is worked on.
template <typename DT, typename XT, int NC, bool RES, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_grad_scalar_kernel(const NormGradArgs a, int group_threads) {
  after_previous();
  extern __shared__ uint4 ring[];
  __shared__ float buf[2][THREADS / 32 * 2];
  const int warps = group_threads >> 5, group = (int)threadIdx.x / group_threads, ngroups = (int)blockDim.x / group_threads;
  const int t = (int)threadIdx.x - group * group_threads;
  const int64_t step = (int64_t)gridDim.x * ngroups, first = (int64_t)blockIdx.x * ngroups + group;
  const int mine = ((int)a.N - t + group_threads - 1) / group_threads;  // values of this thread: t, t + group_threads, ..
  const float inv = 1.0f / (float)a.N;
  float gamma[NC], dg[NC], db[NC];
  DT next_d[NC];
  XT next_x[NC], next_r[RES ? NC : 1];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    gamma[i] = a.gamma && i < mine ? load_as_f32(a.gamma, t + i * group_threads, a.w_bf16) : 1.0f;
    dg[i] = db[i] = 0.0f;
    next_d[i] = from_f32<DT>(0.0f);
    next_x[i] = from_f32<XT>(0.0f);
    if (RES) next_r[i] = from_f32<XT>(0.0f);
  }
  const DT* dy = static_cast<const DT*>(a.dy) + first * a.lddy + t;
  const XT* x = static_cast<const XT*>(a.x) + first * a.ldx + t;
  const XT* res = RES ? static_cast<const XT*>(a.dres) + first * a.lddres + t : nullptr;
  XT* dx = static_cast<XT*>(a.dx) + first * a.lddx + t;
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (i < mine) {
        next_d[i] = dy[i * group_threads];
        next_x[i] = x[i * group_threads];
        if (RES) next_r[i] = res[i * group_threads];
      }
    }
    next_mean = a.mean[r];
    next_rstd = a.rstd[r];
    dy += step * a.lddy;
    x += step * a.ldx;
    if (RES) res += step * a.lddres;
  };
  if (first < a.M) load(first);
  int parity = 0;
  float* my_buf = buf[0] + group * warps * 2;
  for (int64_t r = first; r < a.M; r += step, dx += step * a.lddx) {
    float d[NC], xh[NC], rest[RES ? NC : 1], sums[2] = {0.0f, 0.0f};
    const float mean = next_mean, rstd = next_rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      d[i] = to_f32(next_d[i]);
      xh[i] = to_f32(next_x[i]);
      if (RES) rest[i] = to_f32(next_r[i]);
    }
    if (r + step < a.M) load(r + step);
#pragma unroll
    for (int i = 0; i < NC; ++i) {  // beyond the row dy is 0, so that nothing is added
      xh[i] = (xh[i] - mean) * rstd;
      db[i] += d[i];
      dg[i] = fmaf(d[i], xh[i], dg[i]);
      d[i] *= gamma[i];
      sums[0] += d[i];
      sums[1] = fmaf(d[i], xh[i], sums[1]);
    }
    group_sums_k<2>(sums, my_buf + parity * (THREADS / 32 * 2), warps, group);
    parity ^= 1;
    const float k0 = -sums[0] * inv * rstd, k1 = -sums[1] * inv;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float o = fmaf(fmaf(xh[i], k1, d[i]), rstd, k0);
      if (RES) o += rest[i];
      if (i < mine) dx[i * group_threads] = from_f32<XT>(o);
    }
  }
  if (!a.dgamma && !a.dbeta) return;
  float* out_g = gridDim.x == 1 ? a.dgamma : a.ws + (int64_t)blockIdx.x * 2 * a.N;
  float* out_b = gridDim.x == 1 ? a.dbeta : a.ws + ((int64_t)blockIdx.x * 2 + 1) * a.N;
  float* join = reinterpret_cast<float*>(ring);  // [2][N], as in norm_grad_kernel
  for (int q = 0; q < ngroups; ++q) {
    if (ngroups > 1) __syncthreads();
    if (q != group) continue;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = t + i * group_threads;
      if (i >= mine) continue;
      const float vg = dg[i] + (q > 0 ? join[c] : 0.0f), vb = db[i] + (q > 0 ? join[a.N + c] : 0.0f);
      if (q < ngroups - 1) {
        join[c] = vg;
        join[a.N + c] = vb;
      } else {
        if (out_g) out_g[c] = vg;
        if (out_b) out_b[c] = vb;
      }
    }
  }
}

// ---- rows too long for registers: m0 and m1 of each row, then the columns.

template <typename DT, typename XT>
__global__ void __launch_bounds__(512) row_sums_kernel(const NormGradArgs a, float2* sums) {
  after_previous();
  __shared__ __align__(16) float buf[2][2 * 32];
  int parity = 0;
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const DT* dy = static_cast<const DT*>(a.dy) + r * a.lddy;
    const XT* x = static_cast<const XT*>(a.x) + r * a.ldx;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float v[2] = {0.0f, 0.0f};
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < a.N; c += 512) {
      const float g = to_f32(dy[c]) * (a.gamma ? load_as_f32(a.gamma, c, a.w_bf16) : 1.0f);
      v[0] += g;
      v[1] += g * ((to_f32(x[c]) - mean) * rstd);
    }
    group_sums<false, 2>(v, buf[parity]);
    parity ^= 1;
    if (threadIdx.x == 0) sums[r] = make_float2(v[0] / (float)a.N, v[1] / (float)a.N);
  }
}

// A thread owns V columns of a band of rows.
template <typename DT, typename XT, int V>
__global__ void __launch_bounds__(128) columns_kernel(const NormGradArgs a, const float2* sums, int64_t rows) {
  after_previous();
  const int64_t c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * V;
  if (c >= a.N) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = min(r0 + rows, a.M);
  float w[V], dg[V] = {}, db[V] = {};
  load_weights<V>(a.gamma, a.w_bf16, (int)c, (int)a.N, 1.0f, w);
#pragma unroll 2
  for (int64_t r = r0; r < r1; ++r) {
    float d[V], xh[V], e[V] = {};
    unpack(*reinterpret_cast<const Raw<DT, V>*>(static_cast<const DT*>(a.dy) + r * a.lddy + c), d);
    unpack(*reinterpret_cast<const Raw<XT, V>*>(static_cast<const XT*>(a.x) + r * a.ldx + c), xh);
    if (a.dres) unpack(*reinterpret_cast<const Raw<XT, V>*>(static_cast<const XT*>(a.dres) + r * a.lddres + c), e);
    const float mean = a.mean[r], rstd = a.rstd[r];
    const float2 m = sums[r];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      xh[i] = (xh[i] - mean) * rstd;
      db[i] += d[i];
      dg[i] += d[i] * xh[i];
      e[i] += rstd * (d[i] * w[i] - m.x - xh[i] * m.y);
    }
    *reinterpret_cast<Raw<XT, V>*>(static_cast<XT*>(a.dx) + r * a.lddx + c) = pack(e, Raw<XT, V>());
  }
  float* out_g = gridDim.y == 1 ? a.dgamma : a.ws + (int64_t)blockIdx.y * 2 * a.N;
  float* out_b = gridDim.y == 1 ? a.dbeta : a.ws + ((int64_t)blockIdx.y * 2 + 1) * a.N;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (out_g) out_g[c + i] = dg[i];
    if (out_b) out_b[c + i] = db[i];
  }
}

// `once` blocks or bands of `groups` groups, which take R rows at a time of `rows`: as many times more that no group
// adds more than kMostRows (a multiple of R: 510 or 512), so that the GPU's rounds of blocks stay whole.
int64_t enough(int64_t once, int64_t rows, int groups, int R) {
  const int64_t most = once * groups * (kMostRows / R * R);
  return once * ((rows + most - 1) / most);
}

int64_t bands_of(int64_t M, int64_t N, int V) {
  const int64_t strips = (N + 128 * V - 1) / (128 * V);
  const int64_t once = std::min<int64_t>(std::min<int64_t>(152 * 8 / strips + 1, kMaxBlocks), (M + 15) / 16);
  return std::min<int64_t>(enough(std::max<int64_t>(1, once), M, 1, 1), 65535);  // the grid's limit
}

int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

// Rows of partial sums in the workspace.  Every block or band has a row of the matrix of its own, so that there are
// no more of them than rows (100 MB for one row of 20480 values otherwise); by classes go only more rows than kMaxBlocks.
// `enough` makes fewer than `once` more than the rows need, over all classes kMaxBlocks + (M + 7) / 510.
int64_t most_parts(int64_t M) { return std::min<int64_t>(M, kMaxBlocks + 1 + (M + 7) / 510); }

// `e`: of the launch that leaves the parts.
cudaError_t join(const NormGradArgs& a, int64_t parts, cudaError_t e, cudaStream_t s) {
  if (e != cudaSuccess || parts == 1 || (!a.dgamma && !a.dbeta)) return e;
  return colsum::launch_join<2>(a.ws, (int)parts, a.N, a.dgamma, a.dbeta, s);
}

template <typename DT, typename XT, int NC, int R, int S, int THREADS, int BLOCKS, bool ODD>
cudaError_t run(const NormGradArgs& a, cudaStream_t s) {
  auto kern = a.dres ? norm_grad_kernel<DT, XT, NC, R, S, true, THREADS, BLOCKS, ODD>
                     : norm_grad_kernel<DT, XT, NC, R, S, false, THREADS, BLOCKS, ODD>;
  static BlocksPerSm cache[2];
  const int period = ODD ? row_period(a.ldx) : 1;
  const int group = round32((a.N + (ODD ? 7 : 0) + 8 * NC - 1) / (8 * NC));
  // groups of a block: as many as fit, fewer where that leaves SMs without a block
  const int64_t rows_of_all = (int64_t)152 * R;
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(THREADS / group, (a.M + rows_of_all - 1) / rows_of_all));
  const int threads = group * groups;
  int smem = R * S * NC * threads * (int)(sizeof(Raw<DT, 8>) + sizeof(Raw<XT, 8>) * (a.dres ? 2 : 1));
  smem = std::max(smem, threads * NC * 8 * 8);  // the column sums
  int sms = 0, per_sm = 0;
  const cudaError_t e = cache[a.dres ? 1 : 0].get(kern, threads, smem, sms, per_sm);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)groups * R, of_class = (a.M + period - 1) / period;
  // blocks of a class (`period` divides kMaxBlocks)
  const int64_t once = std::max<int64_t>(1, std::min<int64_t>(kMaxBlocks, (int64_t)sms * per_sm) / period);
  const int64_t blocks = std::min<int64_t>((of_class + rows - 1) / rows, enough(once, of_class, groups, R));
  return join(a, blocks * period, launch_early(kern, dim3((unsigned)(blocks * period)), threads, smem, s, a, group, period), s);
}

template <typename DT, typename XT, int NC, int THREADS, int BLOCKS>
cudaError_t run_scalar(const NormGradArgs& a, cudaStream_t s) {
  auto kern = a.dres ? norm_grad_scalar_kernel<DT, XT, NC, true, THREADS, BLOCKS>
                     : norm_grad_scalar_kernel<DT, XT, NC, false, THREADS, BLOCKS>;
  static BlocksPerSm cache[2];
  const int group = round32((a.N + NC - 1) / NC);
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(THREADS / group, (a.M + 303) / 304));
  const int threads = group * groups, smem = groups > 1 ? (int)(8 * a.N) : 0;
  int sms = 0, per_sm = 0;
  const cudaError_t e = cache[a.dres ? 1 : 0].get(kern, threads, smem, sms, per_sm);
  if (e != cudaSuccess) return e;
  const int64_t once = std::min<int64_t>(kMaxBlocks, (int64_t)sms * per_sm);
  const int64_t blocks = std::min<int64_t>((a.M + groups - 1) / groups, enough(once, a.M, groups, 1));
  return join(a, blocks, launch_early(kern, dim3((unsigned)blocks), threads, smem, s, a, group), s);
}

template <typename DT, typename XT, int V>
cudaError_t run_long(const NormGradArgs& a, cudaStream_t s) {
  const int64_t bands = bands_of(a.M, a.N, V), rows = (a.M + bands - 1) / bands;
  const dim3 grid((unsigned)((a.N + 128 * V - 1) / (128 * V)), (unsigned)((a.M + rows - 1) / rows));
  float2* sums = reinterpret_cast<float2*>(a.ws + most_parts(a.M) * 2 * a.N);
  const dim3 rows_grid((unsigned)std::min<int64_t>(a.M, 152 * 4));
  cudaError_t e = launch_early(row_sums_kernel<DT, XT>, rows_grid, 512, 0, s, a, sums);
  if (e == cudaSuccess) e = launch_early(columns_kernel<DT, XT, V>, grid, 128, 0, s, a, sums, rows);
  return join(a, grid.y, e, s);
}

// The kernel for rows of vectors, or cudaErrorNotSupported where they are too long for it.
template <typename DT, typename XT, bool ODD>
cudaError_t launch_rows(const NormGradArgs& a, cudaStream_t s) {
  const int64_t N = a.N + (ODD ? 7 : 0);                           // columns that a row may touch
  const int64_t bytes = sizeof(DT) + sizeof(XT) * (a.dres ? 2 : 1);  // of a value of the row
  const int64_t group = round32((N + 15) / 16);
  if (N <= 5120) {
    const int64_t row = 320 / group * group * 16 * bytes;  // a row of each group of a block
    // As many rows at a time as two sets of them fit shared memory: the loop's overhead is shared (16384 x 5120
    // bf16 with residual: one row 160 us, two 117, three 108; without it, four rows 89 us, two 103).
    // With few rows one at a time, so that they spread over the SMs.
    // Two blocks per SM where one would have only six warps.
    const bool many = a.M >= 8 * 152;
    if (many && group == 192 && 8 * row <= kRing) return run<DT, XT, 2, 2, 2, 192, 2, ODD>(a, s);
    if (many && group == 192 && 6 * row <= kRing) return run<DT, XT, 2, 1, 3, 192, 2, ODD>(a, s);
    if (many && 8 * row <= kRing) return run<DT, XT, 2, 4, 2, 320, 1, ODD>(a, s);
    if (many && 6 * row <= kRing) return run<DT, XT, 2, 3, 2, 320, 1, ODD>(a, s);
    if (many && 4 * row <= kRing) return run<DT, XT, 2, 2, 2, 320, 1, ODD>(a, s);
    return run<DT, XT, 2, 1, 3, 320, 1, ODD>(a, s);
  }
  if (N <= 10240 && 2 * group * 16 * bytes <= kRing) return run<DT, XT, 2, 1, 2, 640, 1, ODD>(a, s);
  return cudaErrorNotSupported;
}

template <typename DT, typename XT>
cudaError_t launch(const NormGradArgs& a, cudaStream_t s) {
  const bool vec = a.N % 8 == 0 && rows16(a.dy, a.lddy, sizeof(DT)) && rows16(a.x, a.ldx, sizeof(XT)) &&
                   rows16(a.dx, a.lddx, sizeof(XT)) && rows16(a.dres, a.lddres, sizeof(XT)) && rows16(a.gamma, 0, 4);
  if (vec) {
    const cudaError_t e = launch_rows<DT, XT, false>(a, s);
    return e == cudaErrorNotSupported ? run_long<DT, XT, 8>(a, s) : e;
  }
  // Many rows that are long or have a residual: by classes of rows (16384 x 2731 with residual, bf16 72 us against 107
  // value by value, fp32 137 and 156; without it 62 and 72, fp32 108 and 97; 700 x 2001 bf16 11.6 and 10.3).
  const bool bf16_rows = sizeof(DT) == 2 && sizeof(XT) == 2;
  if (a.M >= (a.dres ? 8 : 16) * 152 && (a.dres || a.N > (bf16_rows ? 8 * 192 : 16 * 192)) && rows_shift_as(a.dy, a.lddy, a.ldx) &&
      rows_shift_as(a.x, a.ldx, a.ldx) && rows_shift_as(a.dx, a.lddx, a.ldx) && rows_shift_as(a.dres, a.lddres, a.ldx)) {
    const cudaError_t e = launch_rows<DT, XT, true>(a, s);
    if (e != cudaErrorNotSupported) return e;
  }
  // few rows: more threads to a row, the latency counts; many: fewer, the instructions do (16384 x 2731 fp32 89 us
  // with sixteen values per thread, 180 with eight; 515 x 1023 fp32 9.6 and 6.4 us)
  if (a.M < 8 * 152 && a.N <= 8 * 256) return run_scalar<DT, XT, 8, 256, 2>(a, s);
  if (a.N <= 16 * 192) return run_scalar<DT, XT, 16, 192, 2>(a, s);
  if (a.N <= 16 * 320) return run_scalar<DT, XT, 16, 320, 1>(a, s);
  return run_long<DT, XT, 1>(a, s);
}

}  // namespace
}  // namespace norm

int64_t norm_grad_workspace(int64_t M, int64_t N) {
  // partial column sums of every block or band, and two sums per row
  return norm::most_parts(M) * 2 * N * 4 + (M + 1) / 2 * 2 * 8;
}

cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  using layer::bf16;
  if (a.dy_bf16) return a.x_bf16 ? norm::launch<bf16, bf16>(a, s) : norm::launch<bf16, float>(a, s);
  return a.x_bf16 ? norm::launch<float, bf16>(a, s) : norm::launch<float, float>(a, s);
}

}  // namespace nvfp4
