// linear.cu -- nvfp4_linear: which kernel runs.
#include <algorithm>

#include "layer_internal.h"
#include "linear_launch.h"

namespace nvfp4 {

int64_t linear_workspace(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  if (a.amax) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, 2 * sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  // Tokens in tiles of 128 x 256 features once those fill the GPU; below that the weight's rows take the lanes
  // and K is split until about four blocks per SM share the weight's bytes.
  const int64_t tiles = ((a.M + 127) / 128) * ((a.N + 255) / 256);
  if (a.M > 128 && tiles >= 76) return lin::launch_many(a, s);
  const int bn = a.M <= 16 ? 16 : (a.M <= 32 ? 32 : (a.M <= 64 ? 64 : 128));
  const int64_t blocks = ((a.N + 127) / 128) * ((a.M + bn - 1) / bn), nk = (a.K + 255) / 256;
  int S = 1;
  while (S < 8 && 2 * S <= nk && blocks * S < 4 * 152) S *= 2;
  return lin::launch_split(a, bn, S, s);
}

}  // namespace nvfp4
