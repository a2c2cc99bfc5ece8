// attention_device.cuh -- what the kernels on the cache share: the batch's sequences and
// their places in the cache, checked on the device, where their numbers are.
#pragma once

#include <cstdint>

#include "attention_internal.h"

namespace nvfp4 {
namespace attention {

struct Sequence {
  int first;   // its first row of the call
  int rows;    // how many
  int length;  // tokens in the cache
};

__device__ __forceinline__ void set_status(int* status, int value) {
  if (status) *status = value;  // one of the values that blocks find: they all say what happened
}

// Sequence b if its numbers are in range; no rows and no tokens otherwise.
__device__ __forceinline__ bool load_sequence(const CacheView& c, int b, Sequence& s) {
  const int s0 = c.starts[b], s1 = c.starts[b + 1], n = c.lengths[b];
  if (s0 < 0 || s1 < s0 || s1 > c.T || n < 0 || (int64_t)n > c.table_width * c.page_size) {
    s.first = s.rows = s.length = 0;
    return false;
  }
  s.first = s0;
  s.rows = s1 - s0;
  s.length = n;
  return true;
}

// The last sequence that starts at row t or before it (-1: none), by halving.
__device__ __forceinline__ int find_sequence(const CacheView& c, int t) {
  int lo = -1, hi = c.sequences;  // starts[lo] <= t < starts[hi], with nothing claimed of the ends
  while (hi - lo > 1) {
    const int m = lo + (hi - lo) / 2;
    if (c.starts[m] <= t)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

// Number of the page with position j of sequence b; -1 if it is out of range.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int j) {
  const int p = c.table[(int64_t)b * c.table_stride + j / c.page_size];
  return p >= 0 && p < c.pages ? p : -1;
}

// The batch checked once, by the threads of one block: a call says what is wrong with
// sequences that none of its rows is in, too.
__device__ __forceinline__ void check_batch(const CacheView& c) {
  if (!c.status) return;
  for (int b = threadIdx.x; b < c.sequences; b += blockDim.x) {
    Sequence s;
    if (!load_sequence(c, b, s)) set_status(c.status, NVFP4_ERR_INDEX);
  }
}

}  // namespace attention
}  // namespace nvfp4
