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
// Rows too long for that take two passes: the row sums, then the columns.
#include <algorithm>

#include "column_sums.cuh"
#include "layer_internal.h"
#include "norm_common.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace norm {
namespace {

constexpr int kMaxBlocks = 304;  // two per SM: rows of partial sums in the workspace

// Barrier of a row's group (its threads are whole warps of one block).
__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Two sums over a group of `warps` warps, the same bits in all its threads;
// `buf` (16-byte aligned) is the group's, calls alternate between two of them.
__device__ __forceinline__ void group_sums2(float& a, float& b, float* buf, int warps, int group) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (warps == 1) return;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - group * warps;
  if (lane == 0) {
    buf[2 * warp] = a;
    buf[2 * warp + 1] = b;
  }
  group_sync(1 + group, warps * 32);
  a = b = 0.0f;
  for (int w = 0; w < warps; w += 2) {
    const float4 p = *reinterpret_cast<const float4*>(buf + 2 * w);
    a += p.x;
    b += p.y;
    if (w + 1 < warps) {
      a += p.z;
      b += p.w;
    }
  }
}

// A thread's NC chunks of V values of a row as pairs: neighbours for V = 8,
// values of two chunks for V = 1.
template <typename T, int V, int NC>
struct Row {
  Raw<T, V> raw[NC];
  __device__ __forceinline__ float2 pair(int p) const {
    float2 f[4];
    if constexpr (V == 8) {
      unpack2(raw[p / 4], f);
      return f[p % 4];
    } else {
      return make_float2(to_f32(raw[2 * p].v[0]), to_f32(raw[2 * p + 1].v[0]));
    }
  }
};
// A read of shared memory that the compiler does not merge with an earlier one of the same place.
template <typename R>
__device__ __forceinline__ R reread(const uint8_t* p) {
  R r;
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p));
#pragma unroll
  for (int i = 0; i < (int)sizeof(R) / 16; ++i) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + 16u * i));
    reinterpret_cast<uint4*>(&r)[i] = v;
  }
  return r;
}
// Column of element e of a thread.
template <int V>
__device__ __forceinline__ int column(int t, int group, int e) {
  return V == 8 ? 8 * (t + (e / 8) * group) + e % 8 : t + e * group;
}

// S > 0: S rows of each group on their way in shared memory (16-byte rows, V = 8); S = 0: plain loads.
template <typename DT, typename XT, int V, int NC, int S, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_grad_kernel(const NormGradArgs a, int group_threads) {
  constexpr int P = NC * V / 2;
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) float buf[2][THREADS / 32 * 4];
  const int N = (int)a.N;
  const int warps = group_threads >> 5, group = (int)threadIdx.x / group_threads, ngroups = (int)blockDim.x / group_threads;
  const int t = (int)threadIdx.x - group * group_threads;
  const int64_t step = (int64_t)gridDim.x * ngroups, first = (int64_t)blockIdx.x * ngroups + group;
  const float inv = 1.0f / (float)N;
  const DT* dy = static_cast<const DT*>(a.dy);
  const XT* x = static_cast<const XT*>(a.x);
  const XT* dres = static_cast<const XT*>(a.dres);
  // this thread's slots: stage by stage NC chunks of dy, of x and of dres, each blockDim.x apart
  constexpr int kDy = (int)sizeof(Raw<DT, V>), kX = (int)sizeof(Raw<XT, V>);
  const int stage_bytes = NC * (int)blockDim.x * (kDy + kX * (dres ? 2 : 1));
  uint8_t* slots = reinterpret_cast<uint8_t*>(ring);
  auto slot_dy = [&](int s, int i) { return slots + s * stage_bytes + (i * (int)blockDim.x + (int)threadIdx.x) * kDy; };
  auto slot_x = [&](int s, int i, int which) {
    return slots + s * stage_bytes + NC * (int)blockDim.x * (kDy + which * kX) +
           (i * (int)blockDim.x + (int)threadIdx.x) * kX;
  };
  auto smem = [](const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); };
  auto copy_row = [&](int64_t r, int s) {
    if constexpr (S > 0) {
      if (r < a.M) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = V * (t + i * group_threads);
          copy_chunk<DT>(smem(slot_dy(s, i)), dy + r * a.lddy, c, c < N);
          copy_chunk<XT>(smem(slot_x(s, i, 0)), x + r * a.ldx, c, c < N);
          if (dres) copy_chunk<XT>(smem(slot_x(s, i, 1)), dres + r * a.lddres, c, c < N);
        }
      }
      copies_commit();
    }
  };
  float2 gamma[P], dg[P], db[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c0 = column<V>(t, group_threads, 2 * p), c1 = column<V>(t, group_threads, 2 * p + 1);
    gamma[p].x = a.gamma && c0 < N ? load_as_f32(a.gamma, c0, a.w_bf16) : 1.0f;
    gamma[p].y = a.gamma && c1 < N ? load_as_f32(a.gamma, c1, a.w_bf16) : 1.0f;
    dg[p] = db[p] = splat(0.0f);
  }
#pragma unroll
  for (int s = 0; s < S - 1; ++s) copy_row(first + s * step, s);
  float mean = first < a.M ? a.mean[first] : 0.0f, rstd = first < a.M ? a.rstd[first] : 0.0f;
  int stage = 0, parity = 0;
  float* mine = buf[0] + group * ((warps + 1) & ~1) * 2;
  for (int64_t r = first; r < a.M; r += step) {
    Row<DT, V, NC> rd;
    Row<XT, V, NC> rx, rr;
    auto read = [&]() {  // dy and x of this row (from its slot, they are read again after the sums: registers)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        rd.raw[i] = reread<Raw<DT, V>>(slot_dy(stage, i));
        rx.raw[i] = reread<Raw<XT, V>>(slot_x(stage, i, 0));
      }
    };
    if constexpr (S > 0) {
      copy_row(r + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);  // the slot read in the previous round
      copies_wait<S - 1>();
      read();
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = V * (t + i * group_threads);
        rd.raw[i] = load_chunk<DT, V>(dy + r * a.lddy, c, N);
        rx.raw[i] = load_chunk<XT, V>(x + r * a.ldx, c, N);
        if (dres) rr.raw[i] = load_chunk<XT, V>(dres + r * a.lddres, c, N);
      }
    }
    const float2 scale = splat(rstd), shift = splat(-mean);
    const float rs = rstd;
    if (r + step < a.M) {  // the next row's, long before they are needed
      mean = a.mean[r + step];
      rstd = a.rstd[r + step];
    }
    float2 s0 = splat(0.0f), s1 = splat(0.0f);
#pragma unroll
    for (int p = 0; p < P; ++p) {  // beyond the row dy is 0, so that nothing is added
      const float2 d = rd.pair(p), xh = mul2(add2(rx.pair(p), shift), scale), g = mul2(d, gamma[p]);
      db[p] = add2(db[p], d);
      dg[p] = fma2(d, xh, dg[p]);
      s0 = add2(s0, g);
      s1 = fma2(g, xh, s1);
    }
    float m0 = s0.x + s0.y, m1 = s1.x + s1.y;
    group_sums2(m0, m1, mine + parity * (THREADS / 32 * 4), warps, group);
    parity ^= 1;
    const float2 k1 = splat(-m1 * inv), k0 = splat(-m0 * inv * rs), sc = splat(rs);
    XT* dx = static_cast<XT*>(a.dx) + r * a.lddx;
    if constexpr (S > 0) {
      read();
      if (dres) {
#pragma unroll
        for (int i = 0; i < NC; ++i) rr.raw[i] = *reinterpret_cast<Raw<XT, V>*>(slot_x(stage, i, 1));
      }
      stage = stage == S - 1 ? 0 : stage + 1;
    }
#pragma unroll
    for (int i = 0; i < (V == 8 ? NC : NC / 2); ++i) {
      constexpr int Q = V == 8 ? 4 : 1;  // pairs stored together
      float2 o[Q];
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const int p = i * Q + j;
        const float2 xh = mul2(add2(rx.pair(p), shift), scale);
        o[j] = fma2(fma2(xh, k1, mul2(rd.pair(p), gamma[p])), sc, k0);
        if (dres) o[j] = add2(o[j], rr.pair(p));
      }
      const int c = column<V>(t, group_threads, 2 * i * Q);
      if constexpr (V == 8) {
        if (c < N) *reinterpret_cast<Raw<XT, 8>*>(dx + c) = pack2(o, Raw<XT, 8>());
      } else {
        if (c < N) dx[c] = from_f32<XT>(o[0].x);
        if (c + group_threads < N) dx[c + group_threads] = from_f32<XT>(o[0].y);
      }
    }
  }
  if (!a.dgamma && !a.dbeta) return;
  // one row of column sums per block; alone it is the result
  float* out_g = gridDim.x == 1 ? a.dgamma : a.ws + (int64_t)blockIdx.x * 2 * a.N;
  float* out_b = gridDim.x == 1 ? a.dbeta : a.ws + ((int64_t)blockIdx.x * 2 + 1) * a.N;
  float* join = reinterpret_cast<float*>(ring);  // [2][N]: the groups' sums, added one group after the other
  if (S > 0) copies_wait<0>();
  for (int q = 0; q < ngroups; ++q) {
    if (ngroups > 1) __syncthreads();
    if (q != group) continue;
#pragma unroll
    for (int e = 0; e < NC * V; ++e) {
      const int c = column<V>(t, group_threads, e);
      if (c >= N) continue;
      float vg = e % 2 ? dg[e / 2].y : dg[e / 2].x, vb = e % 2 ? db[e / 2].y : db[e / 2].x;
      if (q > 0) {
        vg += join[c];
        vb += join[N + c];
      }
      if (q < ngroups - 1) {
        join[c] = vg;
        join[N + c] = vb;
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

int64_t bands_of(int64_t M, int64_t N, int V) {
  const int64_t strips = (N + 128 * V - 1) / (128 * V);
  return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(152 * 8 / strips + 1, kMaxBlocks), (M + 15) / 16));
}

int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

cudaError_t join(const NormGradArgs& a, int64_t parts, cudaStream_t s) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || parts == 1 || (!a.dgamma && !a.dbeta)) return e;
  return colsum::launch_join<2>(a.ws, (int)parts, a.N, a.dgamma, a.dbeta, s);
}

template <typename DT, typename XT, int V, int NC, int S, int THREADS, int BLOCKS>
cudaError_t run(const NormGradArgs& a, cudaStream_t s) {
  auto kern = norm_grad_kernel<DT, XT, V, NC, S, THREADS, BLOCKS>;
  const int group = round32((a.N + V * NC - 1) / (V * NC));
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(THREADS / group, (a.M + kMaxBlocks / 2 - 1) / (kMaxBlocks / 2)));
  const int threads = group * groups;
  int smem = S * NC * threads * (int)(sizeof(Raw<DT, V>) + sizeof(Raw<XT, V>) * (a.dres ? 2 : 1));
  if (groups > 1) smem = std::max(smem, (int)(8 * a.N));
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && smem > 40 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = std::min<int64_t>(std::min<int64_t>((a.M + groups - 1) / groups, kMaxBlocks),
                                           (int64_t)sms * std::max(per_sm, 1));
  kern<<<(unsigned)blocks, threads, smem, s>>>(a, group);
  return join(a, blocks, s);
}

template <typename DT, typename XT, int V>
cudaError_t run_long(const NormGradArgs& a, cudaStream_t s) {
  const int64_t bands = bands_of(a.M, a.N, V), rows = (a.M + bands - 1) / bands;
  const dim3 grid((unsigned)((a.N + 128 * V - 1) / (128 * V)), (unsigned)((a.M + rows - 1) / rows));
  float2* sums = reinterpret_cast<float2*>(a.ws + kMaxBlocks * 2 * a.N);
  row_sums_kernel<DT, XT><<<(unsigned)std::min<int64_t>(a.M, 152 * 4), 512, 0, s>>>(a, sums);
  columns_kernel<DT, XT, V><<<grid, 128, 0, s>>>(a, sums, rows);
  return join(a, grid.y, s);
}

template <typename DT, typename XT>
cudaError_t launch(const NormGradArgs& a, cudaStream_t s) {
  const bool vec = a.N % 8 == 0 && rows16(a.dy, a.lddy, sizeof(DT)) && rows16(a.x, a.ldx, sizeof(XT)) &&
                   rows16(a.dx, a.lddx, sizeof(XT)) && rows16(a.dres, a.lddres, sizeof(XT)) && rows16(a.gamma, 0, 4);
  if (vec) {
    constexpr int S = sizeof(XT) == 2 ? 3 : 2;
    if (a.N <= 5120) return run<DT, XT, 8, 2, S, 320, 2>(a, s);
    if (a.N <= 10240) return run<DT, XT, 8, 2, S, 640, 1>(a, s);
    return run_long<DT, XT, 8>(a, s);
  }
  if (a.N <= 2560) return run<DT, XT, 1, 8, 0, 320, 2>(a, s);
  if (a.N <= 5120) return run<DT, XT, 1, 8, 0, 640, 1>(a, s);
  return run_long<DT, XT, 1>(a, s);
}

}  // namespace
}  // namespace norm

int64_t norm_grad_workspace(int64_t M, int64_t N) {
  // partial column sums of every block or band, and two sums per row
  return norm::kMaxBlocks * 2 * N * 4 + (M + 1) / 2 * 2 * 8;
}

cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  using layer::bf16;
  if (a.dy_bf16) return a.x_bf16 ? norm::launch<bf16, bf16>(a, s) : norm::launch<bf16, float>(a, s);
  return a.x_bf16 ? norm::launch<float, bf16>(a, s) : norm::launch<float, float>(a, s);
}

}  // namespace nvfp4
