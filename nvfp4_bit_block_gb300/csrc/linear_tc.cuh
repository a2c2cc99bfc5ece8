// linear_tc.cuh -- what the two kernels of nvfp4_linear share: tensor-core
// steps on NVFP4 stages in shared memory, tensor maps, the epilogue's arithmetic.
//
// A product tile has a "lane" operand of 128 rows (the MMA's M: one TMEM lane
// per row) and a "column" operand of BN rows (the MMA's N: one TMEM column per
// row).  A pipeline stage holds 256 values of K of both: codes in the 128-byte
// swizzle as TMA writes them, and the scales as the quantizer's tiled layout has
// them, 512 bytes per 128 rows and 64 values of K.
#pragma once

#include "layer_device.cuh"
#include "layer_internal.h"
#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace nvfp4 {
namespace lin {

using namespace layer;

constexpr int kBK = 256;           // FP4 values per stage: 128 bytes of codes per row
constexpr int kLaneRows = 128;
constexpr int kLaneTile = kLaneRows * kBK / 2;  // 16 KB
constexpr int kSfBlock = 512;      // scales of 128 rows x 64 values
constexpr int kSfStage = 4 * kSfBlock;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 512 bytes of shared memory (32 rows of 16 bytes) to 4 TMEM columns, repeated
// in the four lane quarters: a block of 128 rows' scales as the block-scaled
// MMA reads them.  Runs in order with the MMAs that the same thread issues.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = tc5::smem_desc(saddr, 0, 128, 0);  // no swizzle, 8-row groups 128 bytes apart
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Number of 64-value groups of K in stage kb (the last stage may be short).
__device__ __forceinline__ int groups_of(int64_t K, int kb) {
  const int64_t left = (K - (int64_t)kb * kBK + 63) / 64;
  return left < 4 ? (int)left : 4;
}

// Issue one stage's loads: codes by TMA (rows and values beyond the operand
// arrive as zeros), the scale blocks that exist by bulk copies.  `bands` is the
// number of 128-row scale bands of the column operand in this tile.
template <int BN>
__device__ __forceinline__ void load_stage(uint32_t st, uint32_t full, const CUtensorMap* lmap, const CUtensorMap* cmap,
                                           const uint8_t* sfl, const uint8_t* sfc, int64_t sf_row, int lrow, int crow,
                                           int kb, int groups, int bands) {
  constexpr int kColTile = BN * kBK / 2;
  const uint32_t sf_bytes = (uint32_t)(groups * kSfBlock);
  tma::arrive_expect_tx(full, (uint32_t)(kLaneTile + kColTile) + sf_bytes * (uint32_t)(1 + bands));
  tma::load_2d(st, lmap, kb * (kBK / 2), lrow, full);
  tma::load_2d(st + kLaneTile, cmap, kb * (kBK / 2), crow, full);
  tc5::bulk_g2s(st + kLaneTile + kColTile, sfl + (int64_t)kb * kSfStage, sf_bytes, full);
  for (int h = 0; h < bands; ++h)
    tc5::bulk_g2s(st + kLaneTile + kColTile + kSfStage * (1 + h), sfc + h * sf_row + (int64_t)kb * kSfStage, sf_bytes,
                  full);
}

// K % 64 == 32: the last group's scales 2 and 3 are padding, whose bytes may be
// anything (NaN times a zero code would be NaN): set them to zero.  The whole
// warp calls this on the stage's scale bands before the tensor cores read them.
__device__ __forceinline__ void clear_tail(uint8_t* sf, int bands, int group, int lane) {
  for (int h = 0; h < bands; ++h) {
    uint4* p = reinterpret_cast<uint4*>(sf + h * kSfStage + group * kSfBlock + 16 * lane);
    uint4 v = *p;
    v.x &= 0xFFFFu;
    v.y &= 0xFFFFu;
    v.z &= 0xFFFFu;
    v.w &= 0xFFFFu;
    *p = v;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// One stage's tensor-core work, issued by one thread: scales to TMEM, then an
// MMA per 64 values of K.  Each stage has TMEM columns of its own for its
// scales: 16 for the lane operand, then 4 per band and group.
template <int BN>
__device__ __forceinline__ void mma_stage(uint32_t acc, uint32_t sf_tmem, uint32_t st, int groups, bool fresh) {
  constexpr uint32_t idesc = tc5::idesc_e2m1_e4m3(kLaneRows, BN);
  constexpr int kBands = (BN + 127) / 128;
  constexpr int kColTile = BN * kBK / 2;
  const uint32_t sf = st + kLaneTile + kColTile;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < groups) {
      copy_scales(sf_tmem + 4u * j, sf + j * kSfBlock);
#pragma unroll
      for (int h = 0; h < kBands; ++h)
        copy_scales(sf_tmem + 16u + 4u * kBands * j + 4u * h, sf + kSfStage * (1 + h) + j * kSfBlock);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < groups) {
      // 64 values = 32 bytes into each 128-byte swizzled row
      const uint64_t ad = tc5::smem_desc(st + 32 * j, 16, 1024, tc5::kLayoutSwizzle128B);
      const uint64_t bd = tc5::smem_desc(st + kLaneTile + 32 * j, 16, 1024, tc5::kLayoutSwizzle128B);
      tc5::mma_nvf4(acc, ad, bd, idesc, sf_tmem + 4u * j, sf_tmem + 16u + 4u * kBands * j, !(fresh && j == 0));
    }
  }
}

// act over a register array, the choice taken once.
template <int NV>
__device__ __forceinline__ void act_all(float* v, int act) {
  switch (act) {
    case NVFP4_ACT_RELU:
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = act_value(v[i], NVFP4_ACT_RELU);
      break;
    case NVFP4_ACT_GELU:
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = act_value(v[i], NVFP4_ACT_GELU);
      break;
    case NVFP4_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = act_value(v[i], NVFP4_ACT_GELU_TANH);
      break;
    case NVFP4_ACT_SILU:
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = act_value(v[i], NVFP4_ACT_SILU);
      break;
    default: break;
  }
}

// Largest magnitude seen by a warp into both entries of the (zeroed) amax pair.
__device__ __forceinline__ void put_amax(float* amax, uint32_t top) {
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(reinterpret_cast<uint32_t*>(amax), top);
    atomicMax(reinterpret_cast<uint32_t*>(amax) + 1, top);
  }
}

}  // namespace lin
}  // namespace nvfp4
