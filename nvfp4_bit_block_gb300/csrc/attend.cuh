// attend.cuh -- what the attention kernels share: which keys a tile of rows sees, and the
// line of work that blocks share out (attend_few.cu).
#pragma once

#include "attention_device.cuh"
#include "launch_early.cuh"
#include "layer_device.cuh"

namespace nvfp4 {
namespace attention {

using bf16 = __nv_bfloat16;
using layer::after_previous;
using layer::launch_early;

// Sequences with one new token and those with few rows (new tokens times the query heads of a key
// head) are attend_few.cu's, the others go to the kernel for many.  Few are at most a.few_rows, and on a
// short context at most kFewShort and a row more for each 16 keys (attend.cu has the reasons).
constexpr int kFewShort = 256;
__device__ __forceinline__ bool is_few(const AttendArgs& a, const Sequence& s) {
  return s.rows <= 1 || (int64_t)s.rows * a.group <= min(a.few_rows, kFewShort + s.length / 16);
}
// What is few by its rows at any length.
inline int64_t surely_few(const AttendArgs& a) { return a.few_rows < kFewShort ? a.few_rows : kFewShort; }

// Whether the query at position p sees key j (0 <= j).
__device__ __forceinline__ bool visible(const AttendArgs& a, const Sequence& s, int p, int j) {
  const bool near = (a.window == 0) | (p - j < a.window) | (j < a.sinks);  // without branches
  return (j < s.length) & (!a.causal | ((j <= p) & near));
}

// The keys that any of a tile of rows sees, in chunks of CH: the first `sinks` chunks, then
// those from `first` on.
template <int CH>
struct Keys {
  int sinks, first, count;  // count: of both
  int all_from, all_to;     // keys that every row sees lie within these (sinks aside)
  int all_sinks;            // .. or below this
  __device__ __forceinline__ int chunk(int i) const { return i < sinks ? i : first + (i - sinks); }
  // steps of four chunks; a tile that sees nothing has one all the same, which writes its zeros
  __device__ __forceinline__ int steps() const { return count <= 4 ? 1 : (count + 3) / 4; }
  // whether every row sees the whole chunk that begins at `key`
  __device__ __forceinline__ bool all_visible(int key) const {
    return key < all_to - (CH - 1) && (key >= all_from || key < all_sinks - (CH - 1));
  }
};

// Rows first_row .. first_row + n - 1 of a sequence's rows of one key head.
template <int CH, typename Index>
__device__ __forceinline__ Keys<CH> rows_keys(const AttendArgs& a, const Sequence& s, Index first_row, int n) {
  Keys<CH> k = {0, 0, 0, 0, s.length, 0};
  int end = s.length;
  if (a.causal) {
    const int before = s.length - s.rows;  // position of the first new token, >= -2^31 + 1
    const int p0 = before + (int)(first_row / (Index)a.group), p1 = before + (int)((first_row + (Index)(n - 1)) / (Index)a.group);
    end = min(end, p1 + 1);
    k.all_to = min(s.length, p0 + 1);
    if (a.window) {
      const int low = (int)max((int64_t)0, (int64_t)p0 - a.window + 1);
      k.all_from = (int)max((int64_t)0, (int64_t)p1 - a.window + 1);
      k.all_sinks = a.sinks;
      k.sinks = (int)(((uint32_t)max(0, min(min(a.sinks, low), end)) + (CH - 1)) / CH);
      k.first = max(low / CH, k.sinks);
    }
  }
  k.count = k.sinks + max(0, (int)(((uint32_t)max(end, 0) + (CH - 1)) / CH) - k.first);
  return k;
}

// Weights are 2^(s - m) with an offset m of the row's own.  m is 7 below the largest score when it moves, and
// moves only where a score passes it by more than 15: weights lie below 2^15, where fp16 still holds them, and
// most steps leave o alone.  As high as that, weights keep their digits down to 2^-21 of the largest and are
// held to 2^-32 of it below; with the maximum itself as m a row with one key far above 65535 others, whose
// value is zero, lost 3 % of its result at e^-17 and all of it at e^-20.
constexpr float kLift = 7.0f, kMoves = 15.0f;

// lse of one row from m and the sum of its weights, -Inf and 0 where it sees nothing.
__device__ __forceinline__ float row_lse(float m, float l) {
  if (l == 0.0f) return -INFINITY;
  return m == -INFINITY ? l : (m + log2f(l)) * 0.6931471805599453f;  // NaN leaves the maximum alone
}
// ---- fp16 products --------------------------------------------------------------------------

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The eight codes of a word as four f16x2 (byte j: its low nibble, then its high one).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t* h) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t scales2(uint32_t two) {  // two scale bytes as f16x2
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// Queries go to fp16 scaled by a power of two per row.  From the bits of the row's largest
// magnitude (they order as the numbers do, NaN above all): what brings it to 2^14 .. 2^15 (bf16's last binade to
// below 2^16, which fp16 holds), and what undoes that.  So high, all eight bits of a value are there down
// to 2^-31 of the largest; with the largest below 4 they went from 2^-18 on.
__device__ __forceinline__ uint32_t query_exponent(uint32_t top) { return min(max(top >> 23, 15u), 253u); }
__device__ __forceinline__ float query_down(uint32_t top) { return __uint_as_float((268u - query_exponent(top)) << 23); }
__device__ __forceinline__ float query_up(uint32_t top) { return __uint_as_float((query_exponent(top) - 14u) << 23); }
__device__ __forceinline__ uint32_t larger_magnitude(uint32_t top, uint32_t two_bf16) {
  return max(top, max(two_bf16 << 16 & 0x7FFF0000u, two_bf16 & 0x7FFF0000u));
}
// Eight queries as they lie in memory; vec: the address is a multiple of 16.
__device__ __forceinline__ uint4 load_query8(const bf16* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
  return make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                    e[6] | (uint32_t)e[7] << 16);
}
__device__ __forceinline__ bool rows_at_16(const Tokens& t) {
  return reinterpret_cast<uintptr_t>(t.p) % 16 == 0 && t.ts % 8 == 0 && t.hs % 8 == 0;
}

// ---- the line of work -----------------------------------------------------------------------

// What a block leaves of the unit that it begins and does not end (last < 0: none).
struct FewHead {
  int last;  // the block that ends it
  int first, head, row, rows;  // the sequence's first row of the call, the key head, the unit's first row and how many
};

// The line cut into G pieces, the first total % G of them a step longer.
struct Pieces {
  int64_t each, longer;
  __device__ __forceinline__ Pieces(int64_t total, int G) {
    if (total <= UINT32_MAX) {  // a division of 64 bits takes about a hundred instructions
      each = (uint32_t)total / (uint32_t)G;
      longer = (uint32_t)total % (uint32_t)G;
    } else {
      each = total / G;
      longer = total % G;
    }
  }
  __device__ __forceinline__ int64_t begin(int64_t i) const { return i * each + (i < longer ? i : longer); }
  __device__ __forceinline__ int holds(int64_t step) const {
    const int64_t cut = longer * (each + 1);
    return (int)(step < cut ? step / (each + 1) : longer + (step - cut) / each);
  }
};

// A line of work along the sequences, `weight(sequence)` units for each: its length, and the
// sequence that unit `mine(length)` of it is in.  Every block adds them up for itself, a
// consecutive part of them in each thread.
struct Line {
  int64_t total;
  int64_t base;  // where `sequence` begins
  int sequence;
  int64_t sums[32];
};
template <int THREADS, typename Weight, typename Mine>
__device__ __forceinline__ void find_line(const CacheView& c, Line& line, Weight weight, Mine mine_of) {
  constexpr int WARPS = THREADS / 32;
  const int t = threadIdx.x, lane = t % 32, warp = t / 32;
  const int64_t each = ((int64_t)c.sequences + THREADS - 1) / THREADS;
  const int64_t from = min((int64_t)c.sequences, t * each), to = min((int64_t)c.sequences, from + each);
  int64_t sum = 0;
  for (int64_t b = from; b < to; ++b) sum += weight((int)b);
  int64_t up = sum;  // with all before
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) line.sums[warp] = up;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i == warp) before = total;
    total += line.sums[i];
  }
  int64_t base = before + up - sum;
  if (t == 0) line.total = total;
  const int64_t mine = mine_of(total);
  if (mine >= base && mine < base + sum) {
    for (int64_t b = from; b < to; ++b) {
      const int64_t n = weight((int)b);
      if (mine < base + n) {
        line.base = base;
        line.sequence = (int)b;
        break;
      }
      base += n;
    }
  }
  __syncthreads();
}

}  // namespace attention

int64_t attend_few_workspace(int64_t T, int group, int dim, int64_t sequences);
cudaError_t launch_attend_few(const AttendArgs& a, cudaStream_t s);
cudaError_t launch_attend_many(const AttendArgs& a, cudaStream_t s);

}  // namespace nvfp4
