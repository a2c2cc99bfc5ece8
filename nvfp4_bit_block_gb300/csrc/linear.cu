// linear.cu -- nvfp4_linear: which kernel runs.
#include "launch_early.cuh"
#include "layer_internal.h"
#include "linear_launch.h"

namespace nvfp4 {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int columns(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

// The weight's rows take the lanes and the tokens one tile of 16, 32 or 64 columns
// or tiles of 128, with K split over the SMs and the pieces joined by a second
// kernel; or, without a second kernel, whole tiles of at most 64 columns where they
// take an SM at most eight steps of K more than its share of the split.
bool whole(int64_t M, int64_t N, int64_t K, int bn) {
  const int64_t steps = ceil_div(K, 256), f = ceil_div(N, 128);
  const int64_t split = ceil_div(f * ceil_div(M, columns(M)) * steps, 152);
  return ceil_div(f * ceil_div(M, bn), 152) * steps <= split + 8;
}
int whole_columns(int64_t M) { return M <= 64 ? columns(M) : 64; }

// More than 128 tokens: by pairs of SMs in tiles of 256 x 256 where that is expected
// to take less time, in ns.  The terms are what calls took: pairs 8.7 us + 0.4 per
// step of K (512 x 5120, K 512 to 8192: 9.6, 12.2, 22.0 us), further rounds of
// tiles 0.5 per step, at least 4.6 (512 x 10240: 14.2, 17.2, 36.0); split with a
// join 8.5 + 0.4 per step of an SM + 0.035 per tile (512 x 5120: K 2048 17.7, 8192
// 26.5; 512 x 2560: 13.2, 18.3); whole tiles 3.5 + 2 per round + 0.26 per step
// (512 x 2560, 5120, 10240, K 512: 8.5, 11.0, 16.2).  Whether an amax is wanted is not
// asked here (the workspace's size does not depend on it), although a call with one
// does not take whole tiles.
bool many(int64_t M, int64_t N, int64_t K) {
  if (M <= 128) return false;
  const int64_t steps = ceil_div(K, 256), f = ceil_div(N, 128), t = f * ceil_div(M, 128);
  const int64_t rounds = ceil_div(ceil_div(M, 256) * ceil_div(N, 256), 76);
  const int64_t more = 800 + 500 * steps, pairs = 8700 + 400 * steps + (rounds - 1) * (more > 4600 ? more : 4600);
  const int64_t turns = ceil_div(f * ceil_div(M, 64), 152);
  return pairs < (whole(M, N, K, whole_columns(M)) ? 3500 + turns * (2000 + 260 * steps)
                                                   : 8500 + 400 * t * steps / 152 + 35 * t);
}

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K) {
  return many(M, N, K) ? 0 : lin::split_workspace(M, N, K, columns(M));
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  if (!many(a.M, a.N, a.K)) {
    const int bn = whole_columns(a.M);
    // an amax is joined by the second kernel
    return !a.amax && whole(a.M, a.N, a.K, bn) ? lin::launch_split(a, bn, true, s) : lin::launch_split(a, columns(a.M), false, s);
  }
  if (a.amax) {
    const cudaError_t e = layer::zero_amax(a.amax, s);
    if (e != cudaSuccess) return e;
  }
  return lin::launch_many(a, s);
}

}  // namespace nvfp4
