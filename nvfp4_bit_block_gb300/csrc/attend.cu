// attend.cu -- attention of a batch's queries to the NVFP4 cache.
//
// For each row (token and query head), with the running maximum m and sum l of a softmax
// over the visible keys j: o = sum exp(s_j - m) v_j / l, lse = m + log l.  Sequences with few
// rows to a key head are bound by the cache's bytes (attend_few.cu), those with many by their
// products (attend_many.cu).  The lengths are on the device: where a batch may hold both, both
// kernels run, and each leaves the other's sequences alone.
//
// What counts as few.  The kernel for many gives 256 rows of a key head to one SM and does not split
// their keys; the one for few takes tiles of 16 rows and deals the keys of all of them out to all SMs,
// at a seventh of the rate for a full 256 rows.  So it is ahead while the tiles,
// over all key heads, are fewer than about 2.1 for each SM.  Measured, few against many, 40 query heads on 8
// of 128 values: one sequence of 65536 keys and 130 rows to a key head 210 and 989 us, 520 rows 714 and 977, 750
// rows 999 and 1000, 1040 rows 1402 and 978; four of 16384 keys and 130 rows each 209 and 266, 180 rows 272 and
// 268, 260 rows 387 and 261; 64 of 4096 keys and 30 rows 213 and 279, 40 rows 290 and 279.  How the rows are spread over
// the sequences only the device knows: if those beyond one token of each make more tiles than that, a sequence
// is few by its even share of the tiles, two at least.  On short contexts the tiles' own cost (about half a
// microsecond for one, to find its place among all) counts more than the keys: with one key head and 2048 rows few
// takes 90 us and many 38 on 1256 keys, with eight and 500 rows 47 and 37 on 1100, 320 rows 36 and 37 on 1064, 520 rows
// 79 and 80 on 4096.  All of T counts, rows behind the last sequence and empty ones too: padding a batch can move a
// sequence to the other kernel, whose roundings differ in their order.  In a batch of next tokens and one long part
// the part is not few and follows the tokens (64 tokens of up to 4096 keys 64 us, 512 on 32768 505, together 589).
#include "attend.cuh"

namespace nvfp4 {

int attend_few_rows(int64_t T, int group, int heads, int64_t sequences) {
  constexpr int64_t kTiles = 320;  // 2.1 * 152
  int64_t tiles = kTiles / heads;
  if (((T - sequences) * group + 15) / 16 * heads > kTiles) tiles = kTiles / (heads * sequences);
  return 16 * (int)(tiles > 2 ? tiles : 2);
}

int64_t attend_workspace(int64_t T, int Hq, int heads, int dim, int64_t sequences) {
  return attend_few_workspace(T, Hq / heads, dim, sequences);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_attend_few(a, s);
  if (e != cudaSuccess || a.c.T <= 1 || (int64_t)a.c.T * a.group <= attention::surely_few(a)) return e;
  return launch_attend_many(a, s);
}

}  // namespace nvfp4
