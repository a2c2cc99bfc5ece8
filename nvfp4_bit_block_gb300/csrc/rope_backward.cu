// rope_backward.cu -- gradient of the norm and rotation of queries and keys.
//
// With g = dy turned back, r = rsqrt(mean(x^2) + eps), xhat = x r and w = g gamma:
//   dx = r (w - xhat mean(w xhat)),   dgamma = sum over tokens and heads of g xhat.
// dy and x are read once and dx is written once, HBM bounds it.  Each block walks over
// groups of tokens, keeps its sums of dgamma in registers and leaves one row of them in
// the workspace; a second kernel adds the rows in order.
// Measured: 16384 tokens x 48 heads x 128 values bf16 145 us, 4.2 TB/s (61 % of the copy rate), fp32 278 us, 4.3 TB/s.
// Issue slots are 52 % busy and DRAM 52 %: angles, weights and sums fill 128 registers, so that an SM holds 16 warps,
// too few for what each waits for (its 420 instructions for four heads, where the arithmetic is 150, follow one
// another through two sums over lanes).  More heads on their way change nothing (147 us with four).
#include <algorithm>
#include <cmath>

#include "column_sums.cuh"
#include "rope_common.cuh"

namespace nvfp4 {
namespace rope {

template <int V, bool INTER, typename TG, typename TX>
__global__ void __launch_bounds__(kThreads, 2) rope_grad_kernel(RopeGradArgs b, int lanes, int tokens, bool gamma_vec,
                                                                int sums) {
  constexpr int SLOTS = slots_of(V);
  // whether the next head's loads are on their way while one is worked on: in bf16 the registers hold both
  constexpr bool AHEAD = sizeof(TG) + sizeof(TX) == 4 && V > 1;
  extern __shared__ unsigned long long turns[];  // rotated; then the angles of two groups, or the sums of eight warps
  const RopeArgs& a = b.r;
  float2* const angles = reinterpret_cast<float2*>(turns + a.rotated);
  after_previous();
  for (int i = threadIdx.x; i < a.rotated; i += kThreads) turns[i] = turns_of(a.inv_freq[i]);
  const Deal at(lanes, tokens);
  const Slots<V, SLOTS, INTER> s(at.lane, lanes, a.D, a.rotated);
  const float share = 1.0f / (float)a.D;
  // queries, then keys: one set of weights and sums at a time
#pragma unroll 1
  for (int keys = blockIdx.y; keys < 2; keys += gridDim.y) {
    const int H = keys ? a.Hk : a.Hq;
    const Tokens in = keys ? a.k : a.q, out = keys ? a.ok : a.oq, xin = keys ? b.xk : b.xq;
    float gamma[SLOTS][2 * V], dg[SLOTS][2 * V] = {};
    load_gamma(s, keys ? a.gamma_k : a.gamma_q, a.w_bf16, gamma_vec, gamma);
    float2* cs = angles;
    __syncthreads();
    RawHead<V, SLOTS, TG> raw_g;
    RawHead<V, SLOTS, TX> raw_x;
    auto fetch = [&](int64_t t, int h) {
      const bool on = t < a.T && h < H;
      raw_g.load(s, on, static_cast<const TG*>(in.p) + t * in.ts + (int64_t)h * in.hs);
      raw_x.load(s, on, static_cast<const TX*>(xin.p) + t * xin.ts + (int64_t)h * xin.hs);
    };
    const int64_t step = (int64_t)gridDim.x * tokens;
    if (AHEAD && H > 0) fetch((int64_t)blockIdx.x * tokens + at.token, at.head);
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; H > 0 && t0 < a.T; t0 += step) {
      const int here = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
      for (int i = threadIdx.x; i < here * a.rotated; i += kThreads)
        cs[i] = angle(a.positions[t0 + i / a.rotated], turns[i % a.rotated], a.turn);
      __syncthreads();
      const int64_t tt = t0 + at.token;
      const bool there = tt < a.T;
      Angles<V, SLOTS> t;
      t.load(s, cs + (there ? at.token * a.rotated : 0));
      cs = cs == angles ? cs + tokens * a.rotated : angles;
#pragma unroll 1
      for (int h = at.head; h - at.head < H; h += at.per) {  // whole warps: lanes of a head share sums
        float g[SLOTS][2 * V], x[SLOTS][2 * V];
        if (!AHEAD) fetch(tt, h);
        raw_g.widen(g);
        raw_x.widen(x);
        if (AHEAD) {
          if (h + at.per - at.head < H)
            fetch(tt, h + at.per);
          else
            fetch(tt + step, at.head);
        }
        if (2 * a.rotated == a.D)
          turn_pairs<true>(s, t, g);
        else
          turn_pairs<false>(s, t, g);
        float2 q2 = make_float2(0.0f, 0.0f), p2 = q2;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; e += 2) {
            const float2 y = two(x[i] + e);
            q2 = fma2(y, y, q2);
            p2 = fma2(mul2(two(g[i] + e), two(gamma[i] + e)), y, p2);
          }
        const float q = lanes_sum(q2.x + q2.y, lanes), p = lanes_sum(p2.x + p2.y, lanes);
        const float rstd = rsqrtf(fmaf(q, share, a.eps));
        if (there && h < H) {
          const float2 r = make_float2(rstd, rstd), along = make_float2(-p * share * rstd * rstd, -p * share * rstd * rstd);
#pragma unroll
          for (int i = 0; i < SLOTS; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; e += 2) {
              const float2 y = two(x[i] + e), z = two(g[i] + e);
              put(dg[i] + e, fma2(z, mul2(y, r), two(dg[i] + e)));
              put(x[i] + e, mul2(r, fma2(y, along, mul2(z, two(gamma[i] + e)))));
            }
          store_head(s, static_cast<TX*>(out.p) + tt * out.ts + (int64_t)h * out.hs, x);
        }
      }
    }
    if (!sums) continue;
    // the lanes of a warp that hold the same values, then the warps one after another
    __syncthreads();
    float* part = reinterpret_cast<float*>(angles);  // [8][D]
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        float v = dg[i][e];
        for (int o = 16; o >= lanes; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        const int d = e < V ? s.first[i] : s.second[i];
        if (d >= 0 && threadIdx.x % 32 < lanes) part[threadIdx.x / 32 * a.D + d + e % V] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) v += part[w * a.D + i];
      b.ws[((int64_t)blockIdx.x * 2 + keys) * a.D + i] = v;
    }
  }
}

// Tokens that a block takes at a time: up to four, so that the blocks of queries and those of keys are all on the GPU
// at once, as far as four will do, and eight of many.  (515 tokens x 12 heads of 96 fp32: 9.3 us; by two, as
// the forward pass takes them, 516 blocks follow each other in two rounds, 11.3.  1000 tokens by eight 11.0 and
// not 13.4, but 700 x 48 heads of 128 bf16 17.0 and not 14.4.)
static int grad_tokens_of(int64_t T) {
  int n = 1;
  while (n < 4 && 2 * T > (int64_t)n * kBlocks) n *= 2;
  return T > 4 * kBlocks ? 8 : n;
}

// Blocks: enough to fill the GPU, and so many that a thread adds at most 512 heads one after
// another.
static int64_t blocks_of(int64_t T, int H) {
  const int tokens = grad_tokens_of(T);
  const int64_t groups = (T + tokens - 1) / tokens, per_group = H;
  return std::min(groups, std::max<int64_t>(kBlocks, (groups * per_group + 511) / 512));
}

template <int V, bool INTER, typename TG, typename TX>
cudaError_t launch(const RopeGradArgs& b, cudaStream_t s) {
  const RopeArgs& a = b.r;
  const int sums = b.dgamma_q || b.dgamma_k, tokens = grad_tokens_of(a.T);
  const int64_t blocks = blocks_of(a.T, std::max(a.Hq, a.Hk));
  const int smem = a.rotated * 8 + std::max(2 * tokens * a.rotated * (int)sizeof(float2), 8 * a.D * (int)sizeof(float));
  const cudaError_t e = launch_early(rope_grad_kernel<V, INTER, TG, TX>, dim3((unsigned)blocks, passes_apart((a.T + tokens - 1) / tokens)), kThreads, smem, s, b,
                                     lanes_of(V, a.D, a.rotated), tokens, gamma_vectors(a, V), sums);
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
