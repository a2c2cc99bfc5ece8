// attend.cu -- attention of a batch's queries to the NVFP4 cache: sequences with few rows go
// to attend_few.cu, the others are taken here.
//
// For each row (token and query head), with the running maximum m and sum l of a softmax
// over the visible keys j: o = sum exp(s_j - m) v_j / l, lse = m + log l.  One block per
// row; its warps take every fourth key, a lane some of a key's values.
#include <cmath>

#include "attend.cuh"

namespace nvfp4 {
namespace attention {

constexpr int kThreads = 128;

__device__ __forceinline__ float cached(const uint8_t* codes, const uint8_t* scales, int d) {
  const float2 v = e2m1x2_values(codes[d / 2]);
  return (d & 1 ? v.y : v.x) * e4m3_value(scales[d / 16]);
}

__global__ void __launch_bounds__(kThreads) attend_kernel(AttendArgs a) {
  __shared__ Sequence seq;
  __shared__ int at;
  __shared__ float ms[4], ls[4], os[4][256];
  const CacheView& c = a.c;
  after_previous();
  const int t = blockIdx.x, h = blockIdx.y, D = c.dim;
  if (threadIdx.x == 0) {
    at = find_sequence(c, t);
    if (at < 0 || !load_sequence(c, at, seq) || t >= seq.first + seq.rows || is_few(a, seq)) at = -1;
  }
  __syncthreads();
  if (at < 0) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n = D / 32, hk = h / a.group;
  const bf16* q = static_cast<const bf16*>(a.q.p) + (int64_t)t * a.q.ts + (int64_t)h * a.q.hs;
  const float f = a.scale * c.alpha[0] * layer::kLog2e;
  float qv[8], o[8] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) qv[i] = i < n ? layer::to_f32(q[lane + 32 * i]) * f : 0.0f;
  const int64_t p = (int64_t)seq.length - seq.rows + (t - seq.first);
  const int64_t end = a.causal ? p + 1 : seq.length;
  for (int64_t j = warp; j < end; j += 4) {
    if (a.window && p - j >= a.window && j >= a.sinks) continue;
    const int page = page_of(c, at, (int)j), row = (int)j % c.page_size;
    if (page < 0) {
      set_status(c.status, NVFP4_ERR_INDEX);
      continue;
    }
    const int64_t co = (int64_t)page * c.cp + (int64_t)hk * c.ch + (int64_t)row * c.cr;
    const int64_t so = (int64_t)page * c.sp + (int64_t)hk * c.sh + (int64_t)row * c.sr;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) s = fmaf(qv[i], cached(c.kc + co, c.ks + so, lane + 32 * i), s);
    s = layer::warp_sum(s);
    const float top = fmaxf(m, s), shrink = m == top ? 1.0f : exp2f(m - top), w = exp2f(s - top);
    m = top;
    l = fmaf(l, shrink, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) o[i] = fmaf(o[i], shrink, w * cached(c.vc + co, c.vs + so, lane + 32 * i));
  }
  if (lane == 0) {
    ms[warp] = m;
    ls[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) os[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float top = ms[0], total = 0.0f, w[4];
#pragma unroll
  for (int i = 1; i < 4; ++i) top = fmaxf(top, ms[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = ms[i] == -INFINITY ? ls[i] : exp2f(ms[i] - top);  // a warp that saw no key, or NaN alone
    total = fmaf(ls[i], w[i], total);
  }
  const bool any = total != 0.0f;
  const float share = any ? c.alpha[1] / total : 0.0f;
  bf16* out = static_cast<bf16*>(a.o.p) + (int64_t)t * a.o.ts + (int64_t)h * a.o.hs;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v = fmaf(os[i][d], w[i], v);
    out[d] = layer::from_f32<bf16>(v * share);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)t * a.Hq + h] = any ? (top + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace attention

int64_t attend_workspace(int64_t, int, int, int dim, int64_t) {
  return attention::few_floats(attention::few_width(dim)) * (int64_t)sizeof(float);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  using namespace attention;
  const cudaError_t e = launch_attend_few(a, s);
  if (e != cudaSuccess || a.c.T <= 1 || (int64_t)a.c.T * a.group <= kFewRows) return e;
  return launch_early(attend_kernel, dim3((unsigned)a.c.T, (unsigned)a.Hq), kThreads, 0, s, a);
}

}  // namespace nvfp4
