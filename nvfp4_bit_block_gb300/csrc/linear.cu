// linear.cu -- nvfp4_linear: which kernel runs.
#include "layer_internal.h"
#include "linear_launch.h"

namespace nvfp4 {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens in tiles of 256 x 256 features once those give every second pair of SMs a
// tile (5120 -> 5120: 512 tokens 16 us, split 20 us; 256 tokens 14 us split);
// below that the weight's rows take the lanes, with the tokens in one tile of 16,
// 32 or 64 columns or in tiles of 128, and K is split over the SMs ..
bool many(int64_t M, int64_t N) { return M > 128 && ceil_div(M, 256) * ceil_div(N, 256) >= 38; }
int columns(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

// .. unless whole tiles take an SM at most eight steps of K more than its share of
// the split, which is what the second kernel costs.  An amax is joined by the
// second kernel.
bool whole(const LinearArgs& a, int bn) {
  const int64_t steps = ceil_div(a.K, 256), f = ceil_div(a.N, 128);
  const int64_t split = ceil_div(f * ceil_div(a.M, columns(a.M)) * steps, 152);
  return !a.amax && ceil_div(f * ceil_div(a.M, bn), 152) * steps <= split + 8;
}

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K) {
  return many(M, N) ? 0 : lin::split_workspace(M, N, K, columns(M));
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  if (!many(a.M, a.N)) {
    const int bn = a.M <= 64 ? columns(a.M) : 64;
    return whole(a, bn) ? lin::launch_split(a, bn, true, s) : lin::launch_split(a, columns(a.M), false, s);
  }
  if (a.amax) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, 2 * sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  return lin::launch_many(a, s);
}

}  // namespace nvfp4
