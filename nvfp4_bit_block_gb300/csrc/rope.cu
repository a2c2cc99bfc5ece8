// rope.cu -- norm of each head's queries and keys and their rotation, in one pass.
//
// For each token and head y = turn(x * rsqrt(mean(x^2) + eps) * gamma): read once and
// written once, HBM bounds it.  A block takes a few tokens: their angles go to shared
// memory once, for all heads.
#include <cmath>

#include "rope_common.cuh"

namespace nvfp4 {
namespace rope {

template <int V, bool INTER, typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int lanes, int tokens) {
  constexpr int SLOTS = slots_of(V);
  extern __shared__ float2 cs[];  // tokens x rotated
  after_previous();
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int here = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
  for (int i = threadIdx.x; i < here * a.rotated; i += kThreads)
    cs[i] = angle(a.positions[t0 + i / a.rotated], a.inv_freq[i % a.rotated], a.turn);
  __syncthreads();
  const int lane = threadIdx.x % lanes, sub = threadIdx.x / lanes, subs = kThreads / lanes;
  const Slots<V, SLOTS, INTER> s(lane, lanes, a.D, a.rotated);
  const float share = 1.0f / (float)a.D;
#pragma unroll 1
  for (int keys = 0; keys < 2; ++keys) {
    const int H = keys ? a.Hk : a.Hq;
    const Tokens in = keys ? a.k : a.q, out = keys ? a.ok : a.oq;
    float gamma[SLOTS][2 * V];
    load_gamma(s, keys ? a.gamma_k : a.gamma_q, a.w_bf16, gamma);
    const int rows = here * H;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += subs) {  // the whole warp stays: lanes of one row share sums
      const int r = r0 + sub;
      const bool on = r < rows;
      const int t = on ? r / H : 0, h = on ? r % H : 0;
      float x[SLOTS][2 * V];
      if (on) {
        load_head(s, static_cast<const TI*>(in.p) + (t0 + t) * in.ts + (int64_t)h * in.hs, x);
      } else {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) x[i][e] = 0.0f;
      }
      if (a.norm) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) q = fmaf(x[i][e], x[i][e], q);
        const float rstd = rsqrtf(fmaf(lanes_sum(q, lanes), share, a.eps));
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) x[i][e] *= rstd * gamma[i][e];
      }
      turn_pairs(s, cs + t * a.rotated, x);
      if (on) store_head(s, static_cast<TO*>(out.p) + (t0 + t) * out.ts + (int64_t)h * out.hs, x);
    }
  }
}

template <int V, bool INTER, typename TI, typename TO>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int tokens = a.T >= 2048 ? 4 : 1;
  const dim3 grid((unsigned)((a.T + tokens - 1) / tokens));
  return launch_early(rope_kernel<V, INTER, TI, TO>, grid, kThreads, tokens * a.rotated * (int)sizeof(float2), s, a,
                      lanes_of(V, a.D, a.rotated), tokens);
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
