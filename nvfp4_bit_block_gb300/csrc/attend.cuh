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

// Sequences with at most this many rows (new tokens times the query heads of a key head) are
// attend_few.cu's, and those with one token; the others go to the kernel for many.
constexpr int kFewRows = 64;

__device__ __forceinline__ bool is_few(const AttendArgs& a, const Sequence& s) {
  return s.rows <= 1 || (int64_t)s.rows * a.group <= kFewRows;
}

// Whether the query at position p sees key j (0 <= j).
__device__ __forceinline__ bool visible(const AttendArgs& a, const Sequence& s, int p, int j) {
  if (j >= s.length) return false;
  if (!a.causal) return true;
  return j <= p && (a.window == 0 || p - j < a.window || j < a.sinks);
}

// The keys that any of a tile of rows sees, in chunks of 16: the first `sinks` chunks, then
// those from `first` on.
struct Keys {
  int sinks, first, count;  // count: of both
  int all_from, all_to;     // keys that every row sees lie within these (sinks aside)
  int all_sinks;            // .. or below this
  __device__ __forceinline__ int chunk(int i) const { return i < sinks ? i : first + (i - sinks); }
  // steps of 64 keys; a tile that sees nothing has one all the same, which writes its zeros
  __device__ __forceinline__ int steps() const { return count <= 4 ? 1 : (count + 3) / 4; }
  __device__ __forceinline__ bool all_visible(int key) const {
    return key + 15 < all_to && (key >= all_from || key + 15 < all_sinks);
  }
};

// Rows first_row .. first_row + n - 1 of a sequence's rows of one key head.
__device__ __forceinline__ Keys rows_keys(const AttendArgs& a, const Sequence& s, int first_row, int n) {
  Keys k = {0, 0, 0, 0, s.length, 0};
  int end = s.length;
  if (a.causal) {
    const int before = s.length - s.rows;  // position of the first new token, >= -2^31 + 1
    const int p0 = before + first_row / a.group, p1 = before + (first_row + n - 1) / a.group;
    end = min(end, p1 + 1);
    k.all_to = min(s.length, p0 + 1);
    if (a.window) {
      const int low = (int)max((int64_t)0, (int64_t)p0 - a.window + 1);
      k.all_from = (int)max((int64_t)0, (int64_t)p1 - a.window + 1);
      k.all_sinks = a.sinks;
      k.sinks = (max(0, min(min(a.sinks, low), end)) + 15) / 16;
      k.first = max(low / 16, k.sinks);
    }
  }
  k.count = k.sinks + max(0, (max(end, 0) + 15) / 16 - k.first);
  return k;
}
__device__ __forceinline__ Keys tile_keys(const AttendArgs& a, const Sequence& s, int tile) {
  return rows_keys(a, s, 16 * tile, min(16, s.rows * a.group - 16 * tile));
}

// o and lse of one row from its sums (unnormalised, to base 2).
__device__ __forceinline__ void finish(const AttendArgs& a, const Sequence& s, int head, int row, int d, float sum,
                                       float top, float l, float alpha_v) {
  const int64_t t = (int64_t)s.first + row / a.group;
  const int h = head * a.group + row % a.group;
  const float share = l != 0.0f ? alpha_v / l : 0.0f;  // nothing seen: zeros
  static_cast<bf16*>(a.o.p)[t * a.o.ts + (int64_t)h * a.o.hs + d] = layer::from_f32<bf16>(sum * share);
  if (d == 0 && a.lse)
    a.lse[t * a.Hq + h] = l != 0.0f ? (top == -INFINITY ? l : (top + log2f(l)) * 0.6931471805599453f) : -INFINITY;
}

// ---- the line of work -----------------------------------------------------------------------

// What a block leaves of the unit that it begins and does not end (last < 0: none).
struct FewHead {
  int last;  // the block that ends it
  int first, head, tile, rows;
};
__device__ __forceinline__ void load_few(const AttendArgs& a, int b, Sequence& s) {
  load_sequence(a.c, b, s);
  if (!is_few(a, s)) s.rows = 0;
}
// Steps of a sequence's tiles of one key head.
__device__ __forceinline__ int64_t sequence_steps(const AttendArgs& a, const Sequence& s) {
  int64_t n = 0;
  for (int r = 0; 16 * r < s.rows * a.group; ++r) n += tile_keys(a, s, r).steps();
  return n;
}

// The line cut into G pieces, the first total % G of them a step longer.
struct Pieces {
  int64_t each, longer;
  __device__ __forceinline__ Pieces(int64_t total, int64_t G) : each(total / G), longer(total % G) {}
  __device__ __forceinline__ int64_t begin(int64_t i) const { return i * each + (i < longer ? i : longer); }
  __device__ __forceinline__ int holds(int64_t step) const {
    const int64_t cut = longer * (each + 1);
    return (int)(step < cut ? step / (each + 1) : longer + (step - cut) / each);
  }
};

// Where the pieces begin: every block adds up the sequences' steps, THREADS of them at a time,
// and finds the sequence that its piece begins in.
struct Line {
  int64_t total;
  int64_t base;  // where `sequence` begins
  int sequence;
  int64_t sums[32];
};
template <int THREADS>
__device__ __forceinline__ void find_line(const AttendArgs& a, Line& line) {
  constexpr int WARPS = THREADS / 32;
  const int t = threadIdx.x, lane = t % 32, warp = t / 32;
  const int64_t each = ((int64_t)a.c.sequences + THREADS - 1) / THREADS;
  const int64_t from = min((int64_t)a.c.sequences, t * each), to = min((int64_t)a.c.sequences, from + each);
  int64_t sum = 0;
  for (int64_t b = from; b < to; ++b) {
    Sequence s;
    load_few(a, (int)b, s);
    sum += sequence_steps(a, s) * a.c.heads;
  }
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
  const int64_t mine = Pieces(total, gridDim.x).begin(blockIdx.x);
  if (mine >= base && mine < base + sum) {
    for (int64_t b = from; b < to; ++b) {
      Sequence s;
      load_few(a, (int)b, s);
      const int64_t n = sequence_steps(a, s) * a.c.heads;
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

// Blocks of attend_few.cu's kernel: as many as an SM holds of them, on every SM.
constexpr int few_per_sm(int DP) { return DP == 64 ? 4 : DP == 128 ? 3 : 2; }
constexpr int few_blocks(int DP) { return 152 * few_per_sm(DP); }
constexpr int few_width(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// The workspace: a FewHead for each block, then two slots (o, m and l of 16 rows) for each.
constexpr int64_t few_slot_floats(int DP) { return 16 * DP + 32; }
constexpr int64_t few_head_floats(int DP) { return (few_blocks(DP) * (int64_t)sizeof(FewHead) / 4 + 3) / 4 * 4; }
constexpr int64_t few_floats(int DP) { return few_head_floats(DP) + 2 * few_blocks(DP) * few_slot_floats(DP); }

}  // namespace attention

cudaError_t launch_attend_few(const AttendArgs& a, cudaStream_t s);

}  // namespace nvfp4
