// cache.cu -- the paged NVFP4 cache of keys and values: tokens quantized as they are
// written, and read back.
//
// Write: for each 16 values x of a head, with b = max |x|,
//   scale = E4M3(b / (6 alpha)),  code = E2M1(x / (scale alpha)).
// Read: code * scale * alpha.  Both move bytes: 2 or 4 per value on one side, 9/16 on
// the other, and HBM bounds them.  A block takes a few tokens; a thread keeps its piece of a
// token (keys or values, head, place in the head) for all of them, so that a token costs it two
// additions for its addresses, and has several on their way.  Where a token lies in the cache is
// found by one thread for each token.
// Measured: 65536 tokens x 8 heads x 128 values of keys and of values read into bf16 60.7 us, 5.7 TB/s
// (83 % of the copy rate); four prompts (23508 tokens) written and read back 57.4 us, 4.3 TB/s, of which
// the write alone 32.5 us, 3.8 TB/s (56 %; fp32 44 us, 5.0 TB/s): issue slots 61 % busy, and a thread's next loads
// begin only when what it has is stored.
#include <cmath>

#include "attention_device.cuh"
#include "launch_early.cuh"
#include "layer_device.cuh"

namespace nvfp4 {
namespace attention {

using layer::after_previous;
using layer::launch_early;
using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;

// Where one token of the call lies: offsets of its row of head 0.
struct Place {
  int64_t codes, scales;
  bool there;        // its page and position are in range
  bool in_sequence;
};

__device__ __forceinline__ Place place_of(const CacheView& c, int t) {
  Place p = {0, 0, false, false};
  const int b = find_sequence(c, t);
  Sequence s;
  if (b < 0 || !load_sequence(c, b, s) || t >= s.first + s.rows) return p;
  p.in_sequence = true;
  const int64_t j = (int64_t)s.length - s.rows + (t - s.first);
  const int page = j >= 0 ? page_of(c, b, (int)j) : -1;
  if (page >= 0) {
    const int row = (int)j % c.page_size;
    p.codes = (int64_t)((uint64_t)page * c.cp + (uint64_t)row * c.cr);
    p.scales = (int64_t)((uint64_t)page * c.sp + (uint64_t)row * c.sr);
    p.there = true;
  } else {
    set_status(c.status, NVFP4_ERR_INDEX);
  }
  return p;
}

// A thread's pieces: of the 2 * heads * pieces that a token has, one in each pass; where a block
// has threads left, they take further tokens.
struct Piece {
  int token, tokens;  // its first token of the block's, and how many the block takes at once
  int piece, head;
  bool values, on;
  __device__ __forceinline__ Piece(int pass, int heads, int pieces) {
    const int all = 2 * heads * pieces;
    tokens = max(1, kThreads / all);
    const int i = pass * kThreads + threadIdx.x;
    token = all <= kThreads ? threadIdx.x / all : 0;
    const int x = all <= kThreads ? threadIdx.x % all : i;
    on = all <= kThreads ? token < tokens : i < all;
    piece = x % pieces;
    const int h = x / pieces;
    values = h >= heads;
    head = values ? h - heads : h;
  }
};
__device__ __forceinline__ int passes_of(int heads, int pieces) { return (2 * heads * pieces + kThreads - 1) / kThreads; }

// 16 values as they lie in memory (bf16: 8 words, fp32: 16).
template <typename T>
struct Block16 {
  uint32_t w[4 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load16(const T* p, bool vec, Block16<T>& r) {
  constexpr int N = 4 * sizeof(T);
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = a.x;
      r.w[4 * i + 1] = a.y;
      r.w[4 * i + 2] = a.z;
      r.w[4 * i + 3] = a.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}
// The largest magnitude; NaN if there is one.
__device__ __forceinline__ float absmax16(const Block16<bf16>& r) {
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = r.w[i];
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m[i]) : "r"(m[i + n]));
  const float a = bf16_lo(m[0] & 0x7FFF7FFFu), b = bf16_hi(m[0] & 0x7FFF7FFFu);
  float t;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(t) : "f"(a), "f"(b));
  return t;
}
__device__ __forceinline__ float absmax16(const Block16<float>& r) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(__uint_as_float(r.w[i]))));
  return m;
}
__device__ __forceinline__ float2 pair16(const Block16<bf16>& r, int i) { return bf16x2_to_f32x2(r.w[i]); }
__device__ __forceinline__ float2 pair16(const Block16<float>& r, int i) {
  return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}

// Codes and scale byte of 16 values.  The quotient x / d is IEEE's: from the rounded reciprocal
// and the remainder (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990: q + r * inv is rounded exactly for a rounded inv), two values at a time.
template <typename T>
__device__ __forceinline__ uint2 quantize16(const Block16<T>& r, float alpha, uint32_t& scale, int* status) {
  constexpr float kMax = 3.402823466e38f;
  float b = absmax16(r);
  const bool odd = !(b <= kMax);  // NaN or Inf: the status says so, NaN becomes 0, Inf the largest number
  if (odd) {
    set_status(status, NVFP4_ERR_NONFINITE);
    b = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = pair16(r, i);
      b = fmaxf(b, fmaxf(fminf(fabsf(x.x), kMax) * (x.x == x.x ? 1.0f : 0.0f), fminf(fabsf(x.y), kMax) * (x.y == x.y ? 1.0f : 0.0f)));
    }
  }
  scale = e4m3_encode(fminf(__fdiv_rn(b, __fmul_rn(6.0f, alpha)), 1.0e6f));
  const float d = __fmul_rn(e4m3_value(scale), alpha);
  const float inv = d > 0.0f ? __frcp_rn(d) : 0.0f;
  const bool far = odd || (d > 0.0f && b > 64.0f * d);  // a saturated scale: quotients that may overflow
  const float2 inv2 = make_float2(inv, inv), nd2 = make_float2(-d, -d);
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 x = pair16(r, i);
    if (far) {
      const float c = 16.0f * d;
      x.x = x.x == x.x ? fminf(fmaxf(x.x, -c), c) : 0.0f;
      x.y = x.y == x.y ? fminf(fmaxf(x.y, -c), c) : 0.0f;
    }
    const float2 q = mul2(x, inv2), e = fma2(fma2(q, nd2, x), inv2, q);
    v[2 * i] = e.x;
    v[2 * i + 1] = e.y;
  }
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) write_kernel(CacheCopyArgs a, int tokens, bool vec) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;  // blocks on their way
  __shared__ Place places[kMaxTokens];
  const CacheView& c = a.c;
  after_previous();
  const float alpha_k = c.alpha[0], alpha_v = c.alpha[1];
  if (!(alpha_k >= 0x1p-100f && alpha_k <= 0x1p100f && alpha_v >= 0x1p-100f && alpha_v <= 0x1p100f)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(c.status, NVFP4_ERR_RANGE);
    return;
  }
  const int t0 = blockIdx.x * tokens, here = min(tokens, c.T - t0), pieces = c.dim / 16;
  const int passes = passes_of(c.heads, pieces);
  bool placed = false;
  for (int pass = 0; pass < passes; ++pass) {
    const Piece w(pass, c.heads, pieces);
    const Tokens& src = w.values ? a.v : a.k;
    const T* p = static_cast<const T*>(src.p) + (int64_t)t0 * src.ts + (int64_t)w.head * src.hs + 16 * w.piece;
    uint8_t* codes = (w.values ? c.vc : c.kc) + (int64_t)w.head * c.ch + 8 * w.piece;
    uint8_t* scales = (w.values ? c.vs : c.ks) + (int64_t)w.head * c.sh + w.piece;
    const float alpha = w.values ? alpha_v : alpha_k;
    for (int k0 = 0; k0 < here; k0 += U * w.tokens) {
      Block16<T> x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = k0 + u * w.tokens + w.token;
        if (w.on && t < here) load16(p + t * src.ts, vec, x[u]);
      }
      if (!placed) {  // while the first values come
        if (threadIdx.x < here) places[threadIdx.x] = place_of(c, t0 + threadIdx.x);
        if (blockIdx.x == 0) check_batch(c);
        __syncthreads();
        placed = true;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = k0 + u * w.tokens + w.token;
        if (!w.on || t >= here || !places[t].there) continue;
        uint32_t scale;
        const uint2 q = quantize16(x[u], alpha, scale, c.status);
        *reinterpret_cast<uint2*>(codes + places[t].codes) = q;
        scales[places[t].scales] = (uint8_t)scale;
      }
    }
  }
}

// A thread's piece is what fills 16 bytes of the result: N codes under one scale.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(CacheCopyArgs a, int tokens, bool vec) {
  constexpr int N = 16 / sizeof(T), U = 4;
  __shared__ Place places[kMaxTokens];
  const CacheView& c = a.c;
  after_previous();
  const int t0 = blockIdx.x * tokens, here = min(tokens, c.T - t0), pieces = c.dim / N;
  if (threadIdx.x < here) places[threadIdx.x] = place_of(c, t0 + threadIdx.x);
  if (blockIdx.x == 0) check_batch(c);
  __syncthreads();
  const int passes = passes_of(c.heads, pieces);
  for (int pass = 0; pass < passes; ++pass) {
    const Piece w(pass, c.heads, pieces);
    const Tokens& dst = w.values ? a.v : a.k;
    if (!w.on || !dst.p) continue;
    T* p = static_cast<T*>(dst.p) + (int64_t)t0 * dst.ts + (int64_t)w.head * dst.hs + N * w.piece;
    const uint8_t* codes = (w.values ? c.vc : c.kc) + (int64_t)w.head * c.ch + N / 2 * w.piece;
    const uint8_t* scales = (w.values ? c.vs : c.ks) + (int64_t)w.head * c.sh + N * w.piece / 16;
    const float alpha = c.alpha[w.values ? 1 : 0];
    for (int k0 = w.token; k0 < here; k0 += U * w.tokens) {
      uint32_t q[U], scale[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = k0 + u * w.tokens;
        q[u] = scale[u] = 0;
        if (t >= here || !places[t].there) continue;
        const uint8_t* from = codes + places[t].codes;
        q[u] = N == 8 ? *reinterpret_cast<const uint32_t*>(from) : *reinterpret_cast<const uint16_t*>(from);
        scale[u] = scales[places[t].scales];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = k0 + u * w.tokens;
        if (t >= here || !places[t].in_sequence) continue;
        const float s = e4m3_value(scale[u]);
        float x[N];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const float2 v = e2m1x2_values(q[u] >> (8 * e) & 0xFFu);
          const float2 y = mul2(mul2(v, make_float2(s, s)), make_float2(alpha, alpha));  // code * scale is exact
          x[2 * e] = y.x;
          x[2 * e + 1] = y.y;
        }
        T* to = p + t * dst.ts;
        if (vec) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (N == 8) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
              o[e] = *reinterpret_cast<const uint32_t*>(&v);
            } else {
              o[e] = __float_as_uint(x[e]);
            }
          }
          *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) to[e] = layer::from_f32<T>(x[e]);
        }
      }
    }
  }
}

// Whether all pieces of k and v begin at 16 bytes.
static bool vectors(const CacheCopyArgs& a) {
  const int64_t n = a.bf16 ? 8 : 4;
  for (const Tokens* t : {&a.k, &a.v})
    if (t->p && (reinterpret_cast<uintptr_t>(t->p) % 16 || t->ts % n || t->hs % n)) return false;
  return true;
}

// Tokens of a block: as many as leave two blocks for each SM.  (At most 4, 8, 16 and 32: four prompts written
// and read back 69, 60, 58 and 62 us, 65536 tokens read 81, 67, 62 and 62.)
static int tokens_of(const CacheView& c) {
  int n = kMaxTokens;
  while (n > 1 && c.T < n * 2 * 152) n /= 2;
  return n;
}

}  // namespace attention

cudaError_t launch_cache_write(const CacheCopyArgs& a, cudaStream_t s) {
  using namespace attention;
  const int n = tokens_of(a.c);
  const dim3 grid((unsigned)((a.c.T - 1) / n + 1));
  return a.bf16 ? launch_early(write_kernel<bf16>, grid, kThreads, 0, s, a, n, vectors(a))
                : launch_early(write_kernel<float>, grid, kThreads, 0, s, a, n, vectors(a));
}
cudaError_t launch_cache_read(const CacheCopyArgs& a, cudaStream_t s) {
  using namespace attention;
  const int n = tokens_of(a.c);
  const dim3 grid((unsigned)((a.c.T - 1) / n + 1));
  return a.bf16 ? launch_early(read_kernel<bf16>, grid, kThreads, 0, s, a, n, vectors(a))
                : launch_early(read_kernel<float>, grid, kThreads, 0, s, a, n, vectors(a));
}

}  // namespace nvfp4
