// rope_common.cuh -- what the norm and rotation of queries and keys shares with its
// gradient: a head's values in the registers of a few lanes, and the angles.
//
// A head is cut into slots of 2 V values, two vectors of V: a slot of the rotated part
// holds V whole pairs (both halves of (i, i + rotated), or 2 V neighbours), so that the
// turn needs no other lane; the rest passes in slots of its own.  Lane l of the L lanes
// that share a head has slots l, l + L, ..  V is the largest number of values that a load
// can take at this alignment.
#pragma once

#include "attention_internal.h"
#include "launch_early.cuh"
#include "layer_device.cuh"

namespace nvfp4 {
namespace rope {

using bf16 = __nv_bfloat16;
using layer::after_previous;
using layer::launch_early;

constexpr int kThreads = 256;

// V values of type T as fp32, and back.
template <int V, typename T>
__device__ __forceinline__ void load_vec(const T* p, float* x) {
  if constexpr (sizeof(T) * V == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
    }
  } else if constexpr (sizeof(T) * V == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    if constexpr (sizeof(T) == 2) {
      x[0] = bf16_lo(w.x);
      x[1] = bf16_hi(w.x);
      x[2] = bf16_lo(w.y);
      x[3] = bf16_hi(w.y);
    } else {
      x[0] = __uint_as_float(w.x);
      x[1] = __uint_as_float(w.y);
    }
  } else if constexpr (sizeof(T) == 2 && V == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    x[0] = bf16_lo(w);
    x[1] = bf16_hi(w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = layer::to_f32(p[i]);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int V, typename T>
__device__ __forceinline__ void store_vec(T* p, const float* x) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                              pack_bf16(x[6], x[7]));
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  } else if constexpr (sizeof(T) == 2 && V == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(x[0], x[1]);
  } else if constexpr (sizeof(T) == 4 && V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else if constexpr (sizeof(T) == 4 && V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = layer::from_f32<T>(x[i]);
  }
}

// Where a lane's slots lie in a head.
template <int V, int SLOTS, bool INTER>
struct Slots {
  int first[SLOTS], second[SLOTS];  // offsets of the slot's two vectors; -1: none
  int pair[SLOTS];                  // first pair of the slot; -1: it passes

  __device__ __forceinline__ Slots(int lane, int lanes, int D, int rotated) {
    const int turned = rotated / V, all = turned + ((D - 2 * rotated) / V + 1) / 2;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int u = lane + i * lanes;
      first[i] = second[i] = pair[i] = -1;
      if (u < turned) {
        first[i] = INTER ? 2 * V * u : V * u;
        second[i] = INTER ? first[i] + V : rotated + V * u;
        pair[i] = V * u;
      } else if (u < all) {
        first[i] = 2 * rotated + 2 * V * (u - turned);
        second[i] = first[i] + V < D ? first[i] + V : -1;
      }
    }
  }
};

// Each slot's 2 V values of a head as they lie in memory, zeros where there are none: loaded
// early, widened when their turn comes.
template <int V, int SLOTS, typename T>
struct RawHead {
  static constexpr int N = V * (int)sizeof(T) >= 4 ? V * (int)sizeof(T) / 4 : 1;  // words of a vector
  uint32_t w[SLOTS][2][N];

  template <bool INTER>
  __device__ __forceinline__ void load(const Slots<V, SLOTS, INTER>& s, bool on, const T* p) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = half ? s.second[i] : s.first[i];
        uint32_t* to = w[i][half];
#pragma unroll
        for (int e = 0; e < N; ++e) to[e] = 0;
        if (!on || at < 0) continue;
        if constexpr (N == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(p + at);
          to[0] = v.x;
          to[1] = v.y;
          to[2] = v.z;
          to[3] = v.w;
        } else if constexpr (N == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p + at);
          to[0] = v.x;
          to[1] = v.y;
        } else if constexpr (V * sizeof(T) == 4) {
          to[0] = *reinterpret_cast<const uint32_t*>(p + at);
        } else {
          to[0] = *reinterpret_cast<const uint16_t*>(p + at);
        }
      }
  }
  __device__ __forceinline__ void widen(float x[SLOTS][2 * V]) const {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (sizeof(T) == 4)
            x[i][half * V + e] = __uint_as_float(w[i][half][e]);
          else
            x[i][half * V + e] = e & 1 ? bf16_hi(w[i][half][e / 2]) : bf16_lo(w[i][half][e / 2]);
        }
  }
};
template <int V, int SLOTS, bool INTER, typename T>
__device__ __forceinline__ void store_head(const Slots<V, SLOTS, INTER>& s, T* p, const float x[SLOTS][2 * V]) {
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    if (s.first[i] >= 0) store_vec<V>(p + s.first[i], x[i]);
    if (s.second[i] >= 0) store_vec<V>(p + s.second[i], x[i] + V);
  }
}
// The same of a head's weights (ones for NULL), whose type is known at run time only; vec: every
// vector of V begins at a multiple of 16 bytes, or of its size.
template <int V, int SLOTS, bool INTER>
__device__ __forceinline__ void load_gamma(const Slots<V, SLOTS, INTER>& s, const void* g, int is_bf16, bool vec,
                                           float x[SLOTS][2 * V]) {
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int at = half ? s.second[i] : s.first[i];
      float* to = x[i] + half * V;
#pragma unroll
      for (int e = 0; e < V; ++e) to[e] = at < 0 ? 0.0f : 1.0f;
      if (at < 0 || !g) continue;
      if (vec && V >= 4) {
        if (is_bf16) {
          load_vec<V>(static_cast<const bf16*>(g) + at, to);
        } else {
#pragma unroll
          for (int e = 0; e < V; e += 4) load_vec<V < 4 ? V : 4>(static_cast<const float*>(g) + at + e, to + e);
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) to[e] = layer::load_as_f32(g, at + e, is_bf16);
      }
    }
}

// Sum over the L lanes (a power of two) that share a head.
__device__ __forceinline__ float lanes_sum(float v, int L) {
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Angles.  With u = frequency / 2 pi in whole turns, position * u modulo 1 depends on u modulo 1
// alone, so u is kept as a 64-bit fraction and the remainder is the product's low 64 bits, for any
// position, negative ones too: exact but for u's own rounding (2^-54, so an angle at position
// 2^31 is off by 2^-21).  In fp32 an angle of 10^6 would be off by 0.03, and a product in fp64 for each
// token and pair took a quarter of the kernel's time (16384 tokens).
__device__ __forceinline__ unsigned long long turns_of(float freq) {
  const double u = (double)freq * 0.15915494309189533577;
  return __double2ull_rz((u - floor(u)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 angle(int position, unsigned long long u, float turn) {
  const long long r = (long long)((unsigned long long)(long long)position * u);
  float s, c;
  sincospif((float)(int)(r >> 32) * 0x1p-31f, &s, &c);  // half turns
  return make_float2(c, s * turn);
}

// A block's place: which token of its group and which of that token's heads a thread begins
// with.  The lanes of a head lie side by side; a token's heads are dealt out to `per` of them.
struct Deal {
  int lane, token, head, per;
  __device__ __forceinline__ Deal(int lanes, int tokens) {
    const int sub = threadIdx.x / lanes;
    per = kThreads / lanes / tokens;
    lane = threadIdx.x % lanes;
    token = sub / per;
    head = sub % per;
  }
};

// The cosines and sines of a lane's pairs: V of each slot.
template <int V, int SLOTS>
struct Angles {
  float c[SLOTS][V], s[SLOTS][V];
  template <bool INTER>
  __device__ __forceinline__ void load(const Slots<V, SLOTS, INTER>& at, const float2* cs) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 t = at.pair[i] >= 0 ? cs[at.pair[i] + e] : make_float2(1.0f, 0.0f);
        c[i][e] = t.x;
        s[i][e] = t.y;
      }
  }
};
// The arithmetic goes two values at a time (packed fp32): with one it kept the issue slots 53 %
// busy and HBM at 70 %.
__device__ __forceinline__ float2 two(const float* x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ void put(float* x, float2 v) {
  x[0] = v.x;
  x[1] = v.y;
}
template <int V, int SLOTS, bool INTER>
__device__ __forceinline__ void turn_slot(const Angles<V, SLOTS>& t, int i, float x[2 * V]) {
  if constexpr (INTER || V == 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 a = two(x + 2 * e), c = make_float2(t.c[i][e], t.c[i][e]), s = make_float2(t.s[i][e], t.s[i][e]);
      put(x + 2 * e, fma2(make_float2(-a.y, a.x), s, mul2(a, c)));
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 a = two(x + e), b = two(x + V + e), c = two(t.c[i] + e), s = two(t.s[i] + e);
      put(x + e, fma2(make_float2(-b.x, -b.y), s, mul2(a, c)));
      put(x + V + e, fma2(a, s, mul2(b, c)));
    }
  }
}
// What passes is left alone: turned by nothing, an infinity in it would reach the value beside it.
// ALL: nothing passes, the same for the whole kernel.  (A lane's own question in every slot costs
// the gradient of 16384 tokens 5 %.)
template <bool ALL, int V, int SLOTS, bool INTER>
__device__ __forceinline__ void turn_pairs(const Slots<V, SLOTS, INTER>& at, const Angles<V, SLOTS>& t,
                                           float x[SLOTS][2 * V]) {
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (ALL || at.pair[i] >= 0) turn_slot<V, SLOTS, INTER>(t, i, x[i]);
}

// Values per vector at these sizes and this alignment: every vector of a slot begins at a
// multiple of its size, so rotated and what passes are multiples of V.  `widest` is 16
// bytes of the wider type.
inline int vector_values(int widest, int D, int rotated, const Tokens* const* t, const int* bytes, int n) {
  for (int V = widest; V > 1; V /= 2) {
    bool ok = rotated % V == 0 && (D - 2 * rotated) % V == 0;
    for (int i = 0; i < n && ok; ++i)
      ok = reinterpret_cast<uintptr_t>(t[i]->p) % (V * bytes[i]) == 0 && t[i]->ts % V == 0 && t[i]->hs % V == 0;
    if (ok) return V;
  }
  return 1;
}

// Lanes that share a head: a power of two that covers its slots, at most a warp.
inline int lanes_of(int V, int D, int rotated) {
  const int slots = rotated / V + ((D - 2 * rotated) / V + 1) / 2;
  int L = 1;
  while (L < slots && L < 32) L *= 2;
  return L;
}
// Tokens that a block takes at a time: up to eight, so that a thread of 8 lanes has every fourth
// head and several on their way; few tokens are spread out, so that no block has two groups.  Where
// few blocks do that, queries and keys go to blocks of their own.  (The gradient, which leaves a row of
// sums for each block, has its own number of tokens.)
constexpr int kBlocks = 152 * 2;
inline int tokens_of(int64_t T) {
  int n = 1;
  while (n < 8 && T > (int64_t)n * kBlocks) n *= 2;
  return n;
}
inline unsigned passes_apart(int64_t groups) { return groups <= kBlocks ? 2 : 1; }
inline bool gamma_vectors(const RopeArgs& a, int V) {
  const uintptr_t n = a.w_bf16 ? 2 * V : 16;
  return reinterpret_cast<uintptr_t>(a.gamma_q) % n == 0 && reinterpret_cast<uintptr_t>(a.gamma_k) % n == 0;
}
// Slots that a lane of a whole warp may have (D <= 512).
constexpr int slots_of(int V) { return V == 8 ? 1 : 8 / V; }

}  // namespace rope
}  // namespace nvfp4
