// linear_launch.h -- launches of nvfp4_linear's kernels, between its translation units.
#pragma once

#include <cuda_runtime.h>

#include "layer_internal.h"

namespace nvfp4 {
namespace lin {

// Few tokens: tiles of 128 features x bn tokens (16, 32, 64 or 128), K split over clusters of S (1, 2, 4 or 8).
cudaError_t launch_split(const LinearArgs& a, int bn, int S, cudaStream_t s);
// Many tokens: persistent tiles of 128 tokens x 256 or 128 features.
cudaError_t launch_many(const LinearArgs& a, cudaStream_t s);

}  // namespace lin
}  // namespace nvfp4
