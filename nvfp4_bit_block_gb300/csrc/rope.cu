// rope.cu -- norm of each head's queries and keys and their rotation, in one pass.
//
// For each token and head y = turn(x * rsqrt(mean(x^2) + eps) * gamma): read once and
// written once, HBM bounds it.  A block walks over groups of a few tokens: their angles go to
// shared memory once for all heads, and a thread keeps those of its pairs for all heads of its
// token.  The next heads' loads are on their way while these are turned, the next group's too.  Queries
// first, then keys: one set of weights at a time.
// Measured: 16384 tokens x 48 heads x 128 values bf16 74.2 us, 5.4 TB/s (80 % of the copy rate), fp32 161 us, 5.0 TB/s.
// Issue slots are 58 % busy, with 16 warps on an SM (120 registers): neither they nor HBM are at their limit.  Four
// heads on their way by asynchronous copies through shared memory change nothing (75.3).
#include <cmath>
#include <type_traits>

#include "rope_common.cuh"

namespace nvfp4 {
namespace rope {

template <int V, bool INTER, typename TI, typename TO>
__global__ void __launch_bounds__(kThreads, 2) rope_kernel(RopeArgs a, int lanes, int tokens, bool gamma_vec) {
  constexpr int SLOTS = slots_of(V);
  constexpr int U = sizeof(TI) == 2 && V > 1 ? 2 : 1;  // heads at a time
  extern __shared__ unsigned long long turns[];  // rotated; then the angles of two groups
  float2* const angles = reinterpret_cast<float2*>(turns + a.rotated);
  float2* cs = angles;
  after_previous();
  const Deal at(lanes, tokens);
  const Slots<V, SLOTS, INTER> s(at.lane, lanes, a.D, a.rotated);
  const float share = 1.0f / (float)a.D;
  const int64_t step = (int64_t)gridDim.x * tokens;
  for (int i = threadIdx.x; i < a.rotated; i += kThreads) turns[i] = turns_of(a.inv_freq[i]);
#pragma unroll 1
  for (int keys = blockIdx.y; keys < 2; keys += gridDim.y) {
    const int H = keys ? a.Hk : a.Hq;
    const Tokens in = keys ? a.k : a.q, out = keys ? a.ok : a.oq;
    RawHead<V, SLOTS, TI> raw[U];
    auto fetch = [&](int64_t t, int h0) {
      const TI* p = static_cast<const TI*>(in.p) + t * in.ts + (int64_t)h0 * in.hs;
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u].load(s, t < a.T && h0 + u * at.per < H, p + (int64_t)(u * at.per) * in.hs);
    };
    if (H > 0) fetch((int64_t)blockIdx.x * tokens + at.token, at.head);
    float gamma[SLOTS][2 * V];
    if (a.norm) load_gamma(s, keys ? a.gamma_k : a.gamma_q, a.w_bf16, gamma_vec, gamma);
    __syncthreads();
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
      for (int h0 = at.head; h0 - at.head < H; h0 += U * at.per) {  // whole warps: lanes of a head share sums
        RawHead<V, SLOTS, TI> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = raw[u];
        if (h0 + U * at.per - at.head < H)
          fetch(tt, h0 + U * at.per);
        else
          fetch(tt + step, at.head);
        TO* to = static_cast<TO*>(out.p) + tt * out.ts + (int64_t)h0 * out.hs;
        auto finish = [&](auto ALL) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float x[SLOTS][2 * V];
            now[u].widen(x);
            if (a.norm) {
              float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int i = 0; i < SLOTS; ++i)
#pragma unroll
                for (int e = 0; e < 2 * V; e += 2) q = fma2(two(x[i] + e), two(x[i] + e), q);
              const float r = rsqrtf(fmaf(lanes_sum(q.x + q.y, lanes), share, a.eps));
#pragma unroll
              for (int i = 0; i < SLOTS; ++i)
#pragma unroll
                for (int e = 0; e < 2 * V; e += 2)
                  put(x[i] + e, mul2(two(x[i] + e), mul2(two(gamma[i] + e), make_float2(r, r))));
            }
            turn_pairs<ALL.value>(s, t, x);
            if (there && h0 + u * at.per < H) store_head(s, to + (int64_t)(u * at.per) * out.hs, x);
          }
        };
        if (2 * a.rotated == a.D)
          finish(std::true_type());
        else
          finish(std::false_type());
      }
    }
  }
}

template <int V, bool INTER, typename TI, typename TO>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int lanes = lanes_of(V, a.D, a.rotated), tokens = tokens_of(a.T);
  const int64_t groups = (a.T + tokens - 1) / tokens;
  const int smem = a.rotated * (8 + 2 * tokens * (int)sizeof(float2));
  return launch_early(rope_kernel<V, INTER, TI, TO>, dim3((unsigned)(groups < kBlocks ? groups : kBlocks), passes_apart(groups)), kThreads, smem,
                      s, a, lanes, tokens, gamma_vectors(a, V));
}

template <typename TI, typename TO>
cudaError_t by_width(const RopeArgs& a, cudaStream_t s) {
  constexpr int bi = sizeof(TI), bo = sizeof(TO), widest = 16 / (bi > bo ? bi : bo);
  const Tokens* t[4] = {&a.q, &a.k, &a.oq, &a.ok};
  const int bytes[4] = {bi, bi, bo, bo};
  const int V = vector_values(widest, a.D, a.rotated, t, bytes, 4);
  if constexpr (widest == 8) {
    if (V == 8) return a.interleaved ? launch<8, true, TI, TO>(a, s) : launch<8, false, TI, TO>(a, s);
  }
  if (V == 4) return a.interleaved ? launch<4, true, TI, TO>(a, s) : launch<4, false, TI, TO>(a, s);
  if (V == 2) return a.interleaved ? launch<2, true, TI, TO>(a, s) : launch<2, false, TI, TO>(a, s);
  return a.interleaved ? launch<1, true, TI, TO>(a, s) : launch<1, false, TI, TO>(a, s);
}

}  // namespace rope

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  using namespace rope;
  if (a.in_bf16) return a.out_bf16 ? by_width<bf16, bf16>(a, s) : by_width<bf16, float>(a, s);
  return a.out_bf16 ? by_width<float, bf16>(a, s) : by_width<float, float>(a, s);
}

}  // namespace nvfp4
