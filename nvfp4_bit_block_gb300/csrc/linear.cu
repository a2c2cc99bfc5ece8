// linear.cu -- nvfp4_linear: which kernel runs.
#include "layer_internal.h"
#include "linear_launch.h"

namespace nvfp4 {
namespace {

// Tokens in tiles of 256 x 256 features once those give most SM pairs a tile;
// below that the weight's rows take the lanes and K is split over the SMs, with
// the tokens in one tile of 16, 32 or 64 columns or in tiles of 128.
bool many(int64_t M, int64_t N) { return M > 128 && ((M + 255) / 256) * ((N + 255) / 256) >= 38; }
int columns(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K) {
  return many(M, N) ? 0 : lin::split_workspace(M, N, K, columns(M));
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  if (!many(a.M, a.N)) return lin::launch_split(a, columns(a.M), s);
  if (a.amax) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, 2 * sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  return lin::launch_many(a, s);
}

}  // namespace nvfp4
