// rope_backward.cu -- gradient of the norm and rotation of queries and keys.
//
// With g = dy turned back, r = rsqrt(mean(x^2) + eps), xhat = x r and w = g gamma:
//   dx = r (w - xhat mean(w xhat)),   dgamma = sum over tokens and heads of g xhat.
// dy and x are read once and dx is written once, HBM bounds it.  Each block walks over
// groups of tokens, keeps its sums of dgamma in registers and leaves one row of them in
// the workspace; a second kernel adds the rows in order.
#include <algorithm>
#include <cmath>

#include "column_sums.cuh"
#include "rope_common.cuh"

namespace nvfp4 {
namespace rope {

template <int V, bool INTER, typename TG, typename TX>
__global__ void __launch_bounds__(kThreads) rope_grad_kernel(RopeGradArgs b, int lanes, int tokens, int sums) {
  constexpr int SLOTS = slots_of(V);
  extern __shared__ float2 cs[];  // tokens x rotated, then the sums of eight warps
  const RopeArgs& a = b.r;
  after_previous();
  const int lane = threadIdx.x % lanes, sub = threadIdx.x / lanes, subs = kThreads / lanes;
  const Slots<V, SLOTS, INTER> s(lane, lanes, a.D, a.rotated);
  const float share = 1.0f / (float)a.D;
  float dg[2][SLOTS][2 * V] = {};
  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
    const int here = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
    for (int i = threadIdx.x; i < here * a.rotated; i += kThreads)
      cs[i] = angle(a.positions[t0 + i / a.rotated], a.inv_freq[i % a.rotated], a.turn);
    __syncthreads();
#pragma unroll
    for (int keys = 0; keys < 2; ++keys) {
      const int H = keys ? a.Hk : a.Hq;
      const Tokens in = keys ? a.k : a.q, out = keys ? a.ok : a.oq, xin = keys ? b.xk : b.xq;
      float gamma[SLOTS][2 * V];
      load_gamma(s, keys ? a.gamma_k : a.gamma_q, a.w_bf16, gamma);
      const int rows = here * H;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += subs) {
        const int r = r0 + sub;
        const bool on = r < rows;
        const int t = on ? r / H : 0, h = on ? r % H : 0;
        float g[SLOTS][2 * V], x[SLOTS][2 * V];
        if (on) {
          load_head(s, static_cast<const TG*>(in.p) + (t0 + t) * in.ts + (int64_t)h * in.hs, g);
          load_head(s, static_cast<const TX*>(xin.p) + (t0 + t) * xin.ts + (int64_t)h * xin.hs, x);
        } else {
#pragma unroll
          for (int i = 0; i < SLOTS; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) g[i][e] = x[i][e] = 0.0f;
        }
        turn_pairs(s, cs + t * a.rotated, g);
        float q = 0.0f, p = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            q = fmaf(x[i][e], x[i][e], q);
            p = fmaf(g[i][e] * gamma[i][e], x[i][e], p);
          }
        q = lanes_sum(q, lanes);
        p = lanes_sum(p, lanes);
        const float rstd = rsqrtf(fmaf(q, share, a.eps));
        const float along = p * share * rstd * rstd;
        if (on) {
#pragma unroll
          for (int i = 0; i < SLOTS; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
              dg[keys][i][e] = fmaf(g[i][e], x[i][e] * rstd, dg[keys][i][e]);
              x[i][e] = rstd * (g[i][e] * gamma[i][e] - x[i][e] * along);
            }
          store_head(s, static_cast<TX*>(out.p) + (t0 + t) * out.ts + (int64_t)h * out.hs, x);
        }
      }
    }
    __syncthreads();
  }
  if (!sums) return;
  // the lanes of a warp that hold the same values, then the warps one after another
  float* part = reinterpret_cast<float*>(cs);  // [8][2][D]
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int keys = 0; keys < 2; ++keys)
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        float v = dg[keys][i][e];
        for (int o = 16; o >= lanes; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        const int at = e < V ? s.first[i] : s.second[i];
        if (at >= 0 && threadIdx.x % 32 < lanes) part[(warp * 2 + keys) * a.D + at + e % V] = v;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += part[w * 2 * a.D + i];
    b.ws[(int64_t)blockIdx.x * 2 * a.D + i] = v;
  }
}

// Tokens that a block takes at a time, and blocks: enough to fill the GPU, and so many that
// a thread adds at most 512 heads one after another.
constexpr int kTokens = 4;
constexpr int kBlocks = 152 * 4;
static int64_t blocks_of(int64_t T, int H) {
  const int64_t groups = (T + kTokens - 1) / kTokens;
  // a group's heads are spread over at least 8 rows of lanes
  const int64_t per_group = ((int64_t)kTokens * H + 7) / 8;
  const int64_t few = (groups * per_group + 511) / 512;
  return std::min(groups, std::max<int64_t>(kBlocks, few));
}

template <int V, bool INTER, typename TG, typename TX>
cudaError_t launch(const RopeGradArgs& b, cudaStream_t s) {
  const RopeArgs& a = b.r;
  const int sums = b.dgamma_q || b.dgamma_k;
  const int64_t blocks = blocks_of(a.T, std::max(a.Hq, a.Hk));
  const int smem = std::max(kTokens * a.rotated * (int)sizeof(float2), 8 * 2 * a.D * (int)sizeof(float));
  const cudaError_t e = launch_early(rope_grad_kernel<V, INTER, TG, TX>, dim3((unsigned)blocks), kThreads, smem, s, b,
                                     lanes_of(V, a.D, a.rotated), kTokens, sums);
  if (e != cudaSuccess || !sums) return e;
  return colsum::launch_join<2>(b.ws, (int)blocks, a.D, b.dgamma_q, b.dgamma_k, s);
}

template <typename TG, typename TX>
cudaError_t by_width(const RopeGradArgs& b, cudaStream_t s) {
  constexpr int bg = sizeof(TG), bx = sizeof(TX), widest = 16 / (bg > bx ? bg : bx);
  const RopeArgs& a = b.r;
  const Tokens* t[6] = {&a.q, &a.k, &a.oq, &a.ok, &b.xq, &b.xk};
  const int bytes[6] = {bg, bg, bx, bx, bx, bx};
  const int V = vector_values(widest, a.D, a.rotated, t, bytes, 6);
  if constexpr (widest == 8) {
    if (V == 8) return a.interleaved ? launch<8, true, TG, TX>(b, s) : launch<8, false, TG, TX>(b, s);
  }
  if (V == 4) return a.interleaved ? launch<4, true, TG, TX>(b, s) : launch<4, false, TG, TX>(b, s);
  if (V == 2) return a.interleaved ? launch<2, true, TG, TX>(b, s) : launch<2, false, TG, TX>(b, s);
  return a.interleaved ? launch<1, true, TG, TX>(b, s) : launch<1, false, TG, TX>(b, s);
}

}  // namespace rope

int64_t rope_grad_workspace(int64_t T, int Hq, int Hk, int D) {
  return rope::blocks_of(T, std::max(Hq, Hk)) * 2 * D * (int64_t)sizeof(float);
}

cudaError_t launch_rope_grad(const RopeGradArgs& b, cudaStream_t s) {
  using namespace rope;
  const RopeArgs& a = b.r;
  if (a.in_bf16) return a.out_bf16 ? by_width<bf16, bf16>(b, s) : by_width<bf16, float>(b, s);
  return a.out_bf16 ? by_width<float, bf16>(b, s) : by_width<float, float>(b, s);
}

}  // namespace nvfp4
