// linear_launch.h -- launches of nvfp4_linear's kernels, between its translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "layer_internal.h"

namespace nvfp4 {
namespace lin {

// Few tokens: tiles of 128 features x bn tokens (16, 32, 64 or 128), K split over clusters of S (1, 2, 4 or 8).
cudaError_t launch_split(const LinearArgs& a, int bn, int S, cudaStream_t s);
// Many tokens: pairs of blocks walk tiles of 256 tokens x 256 features.
cudaError_t launch_many(const LinearArgs& a, cudaStream_t s);

// rows x cols elements (row stride ld; 16-byte aligned rows) in boxes of 64 bytes x box_rows, 64-byte swizzle.
// NULL gives an empty map.
cudaError_t make_out_map(CUtensorMap* map, const void* p, bool is_bf16, int64_t rows, int64_t cols, int64_t ld,
                         int box_rows);

}  // namespace lin
}  // namespace nvfp4
