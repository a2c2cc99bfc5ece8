// out_tmap.cu -- host-side tensor maps of nvfp4_linear's dense matrices (d, z, residual).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstring>

#include "linear_launch.h"

namespace nvfp4 {
namespace lin {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 load_encoder() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

}  // namespace

cudaError_t make_out_map(CUtensorMap* map, const void* p, bool is_bf16, int64_t rows, int64_t cols, int64_t ld,
                         int box_rows) {
  std::memset(map, 0, sizeof(*map));
  if (!p) return cudaSuccess;  // not used
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = load_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t size = is_bf16 ? 2 : 4;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * size};
  const cuuint32_t box[2] = {(cuuint32_t)(64 / size), (cuuint32_t)box_rows};
  const cuuint32_t elem_strides[2] = {1u, 1u};
  const CUresult r =
      encode(map, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
             const_cast<void*>(p), dims, strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace lin
}  // namespace nvfp4
