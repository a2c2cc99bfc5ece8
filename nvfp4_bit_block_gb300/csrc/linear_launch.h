// linear_launch.h -- launches of nvfp4_linear's kernels, between its translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "layer_internal.h"

namespace nvfp4 {
namespace lin {

// Few tokens: tiles of 128 features x bn tokens.  Either K is split over the SMs (bn 16, 32 or 64 for at most as many
// tokens, else 128; split_workspace bytes at a.ws; amax), or the tiles are whole (bn 16 or 32 for at most as many
// tokens, else 64; no workspace, no amax).
cudaError_t launch_split(const LinearArgs& a, int bn, bool whole, cudaStream_t s);
int64_t split_workspace(int64_t M, int64_t N, int64_t K, int bn);
// Many tokens: pairs of blocks walk tiles of 256 tokens x 256 features.
cudaError_t launch_many(const LinearArgs& a, cudaStream_t s);

// rows x cols elements (row stride ld; 16-byte aligned rows) in boxes of 64 bytes x box_rows, 64-byte swizzle.
// NULL gives an empty map.
cudaError_t make_out_map(CUtensorMap* map, const void* p, bool is_bf16, int64_t rows, int64_t cols, int64_t ld,
                         int box_rows);

}  // namespace lin
}  // namespace nvfp4
