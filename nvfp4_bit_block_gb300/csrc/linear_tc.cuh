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

// ---- pairs of blocks (cta_group::2): the two blocks of a cluster of two form one
// MMA of 256 rows; each holds its 128 rows of the lane operand, half of the column
// operand's rows, its 128 rows of the accumulator, and all of the column scales.
__device__ __forceinline__ void alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma2_nvf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// The mbarrier at this offset in both blocks receives an arrival when the pair's MMAs issued so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrival on the barrier at this offset in block `rank` of the cluster, and the
// wait for such arrivals.  What they order is tensor-core work (TMEM accesses,
// fenced by tcgen05.fence, and tiles whose copies have completed), no ordinary
// memory, so the arrival has the default scope: a release at cluster scope made
// a stage of the pair kernel take 1930 instead of 930 clocks.
__device__ __forceinline__ void arrive_at(uint32_t bar, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(bar), "r"(rank));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < tma::kWaitLimitPolls; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (i == 0) t0 = tma::globaltimer();
    if ((i & 255u) == 255u && tma::globaltimer() - t0 > tma::kWaitLimitNs) return false;
  }
  return false;
}

// ---- stores of staged tiles by TMA, tracked in bulk groups of the issuing thread.  A
// row of the tensor is written in whole pieces of 16 bytes: it has to end at one.
__device__ __forceinline__ void store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void stores_read() {  // all but the LEFT latest stores have read shared memory
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// K in stages of 256 values: how many, the 64-value groups of the last one, and
// whether its last group is half padding (K % 64 == 32).
struct Steps {
  int n, last;
  bool tail;
  __device__ __forceinline__ explicit Steps(int64_t K)
      : n((int)((K + kBK - 1) / kBK)), last((int)((K - (int64_t)(n - 1) * kBK + 63) / 64)), tail(K % 64 != 0) {}
  __device__ __forceinline__ int groups(int kb) const { return kb == n - 1 ? last : 4; }
};

// A position in a ring of N slots: the slot and the parity of the use that it is in.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Test builds whose copies are armed but never issued, so that every wait runs out.
#ifdef NVFP4_TEST_NO_COPIES
constexpr bool kCopies = false;
#else
constexpr bool kCopies = true;
#endif

// Issue the loads of one stage's codes (rows and values beyond the operand
// arrive as zeros) and of the scale blocks that exist: the lane operand's 128
// rows, then `bands` bands of the column operand.
__device__ __forceinline__ void load_codes(uint32_t st, uint32_t full, const CUtensorMap* lmap, const CUtensorMap* cmap,
                                           int lrow, int crow, int kb) {
  if (!kCopies) return;
  tma::load_2d(st, lmap, kb * (kBK / 2), lrow, full);
  tma::load_2d(st + kLaneTile, cmap, kb * (kBK / 2), crow, full);
}
__device__ __forceinline__ void load_scales(uint32_t sf, uint32_t full, const uint8_t* sfl, const uint8_t* sfc,
                                            int64_t sf_row, int kb, int groups, int bands) {
  if (!kCopies) return;
  const uint32_t bytes = (uint32_t)(groups * kSfBlock);
  tc5::bulk_g2s(sf, sfl + (int64_t)kb * kSfStage, bytes, full);
  for (int h = 0; h < bands; ++h)
    tc5::bulk_g2s(sf + kSfStage * (1 + h), sfc + h * sf_row + (int64_t)kb * kSfStage, bytes, full);
}

// One stage's scales by the four warps of TMEM's lane quarters: each lane holds
// the 16 bytes of its row of a block, and every quarter gets the same ones.
// `tail`: the last group's scales 2 and 3 are padding and become zeros.
template <int BANDS>
__device__ __forceinline__ void put_scales(uint32_t sf_tmem, const uint8_t* sf, int groups, bool tail, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 v[1 + BANDS];
#pragma unroll
    for (int h = 0; h < 1 + BANDS; ++h)
      v[h] = *reinterpret_cast<const uint4*>(sf + h * kSfStage + j * kSfBlock + 16 * lane);
    if (tail && j == groups - 1) {
#pragma unroll
      for (int h = 0; h < 1 + BANDS; ++h) {
        v[h].x &= 0xFFFFu;
        v[h].y &= 0xFFFFu;
        v[h].z &= 0xFFFFu;
        v[h].w &= 0xFFFFu;
      }
    }
    tc5::st_32x32b_x4(sf_tmem + 4u * j, v[0]);
#pragma unroll
    for (int h = 0; h < BANDS; ++h) tc5::st_32x32b_x4(sf_tmem + 16u + 4u * BANDS * j + 4u * h, v[1 + h]);
  }
  tc5::wait_st();
}

// Shared-memory descriptors of a stage's two tiles; 64 values of K are 32 bytes
// (2 descriptor units) into each 128-byte swizzled row.
struct StageDesc {
  uint64_t lane, col;
  __device__ __forceinline__ explicit StageDesc(uint32_t st)
      : lane(tc5::smem_desc(st, 16, 1024, tc5::kLayoutSwizzle128B)),
        col(tc5::smem_desc(st + kLaneTile, 16, 1024, tc5::kLayoutSwizzle128B)) {}
};

// One stage's tensor-core work, issued by one thread: an MMA per 64 values of K.
// Each stage has TMEM columns of its own for its scales: 16 for the lane
// operand, then 4 per band and group.  A whole stage is straight-line code: a
// branch before each MMA kept the tensor pipe waiting for its next instruction
// (16384 x 5120 x 20480: 714 us with, 627 us without).
// `shift`: the column operand's rows begin at row 32 * shift of their 128-row
// band, whose scales TMEM holds 32 rows to a column.
template <int BN>
__device__ __forceinline__ void mma_step(uint32_t acc, uint32_t sf_tmem, uint32_t shift, StageDesc d, int j, bool add) {
  constexpr uint32_t idesc = tc5::idesc_e2m1_e4m3(kLaneRows, BN);
  constexpr int kBands = (BN + 127) / 128;
  tc5::mma_nvf4(acc, d.lane + 2 * j, d.col + 2 * j, idesc, sf_tmem + 4u * j, sf_tmem + 16u + 4u * kBands * j + shift, add);
}
template <int BN>
__device__ __forceinline__ void mma_stage(uint32_t acc, uint32_t sf_tmem, uint32_t shift, StageDesc d, int groups,
                                          bool fresh) {
  if (groups == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) mma_step<BN>(acc, sf_tmem, shift, d, j, j > 0 || !fresh);
  } else {
    for (int j = 0; j < groups; ++j) mma_step<BN>(acc, sf_tmem, shift, d, j, j > 0 || !fresh);
  }
}

// The same for a pair of blocks: 256 rows of lanes, BN columns of which each block holds half.
template <int BN>
__device__ __forceinline__ void mma2_step(uint32_t acc, uint32_t sf_tmem, StageDesc d, int j, bool add) {
  constexpr uint32_t idesc = tc5::idesc_e2m1_e4m3(2 * kLaneRows, BN);
  constexpr int kBands = (BN + 127) / 128;
  mma2_nvf4(acc, d.lane + 2 * j, d.col + 2 * j, idesc, sf_tmem + 4u * j, sf_tmem + 16u + 4u * kBands * j, add);
}
template <int BN>
__device__ __forceinline__ void mma2_stage(uint32_t acc, uint32_t sf_tmem, StageDesc d, int groups, bool fresh) {
  if (groups == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) mma2_step<BN>(acc, sf_tmem, d, j, j > 0 || !fresh);
  } else {
    for (int j = 0; j < groups; ++j) mma2_step<BN>(acc, sf_tmem, d, j, j > 0 || !fresh);
  }
}

// act on pairs with the packed fp32 instructions: the operations of act_value in
// its order, so with its results.
__device__ __forceinline__ float2 splat2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 gate2(float2 z, float2 neg) {  // z / (1 + 2^neg)
  const float2 e = add2(make_float2(ex2(neg.x), ex2(neg.y)), splat2(1.0f));
  return mul2(z, make_float2(rcp(e.x), rcp(e.y)));
}
template <int ACT, typename T>
__device__ __forceinline__ float2 act_pair(float2 z) {
  if constexpr (ACT == NVFP4_ACT_RELU) {
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(z.x) : "f"(z.x));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(z.y) : "f"(z.y));
    return z;
  } else if constexpr (ACT == NVFP4_ACT_GELU_TANH) {
    return gate2(z, mul2(z, fma2(mul2(z, z), splat2(-kLog2e * kGeluC * kGeluA), splat2(-kLog2e * kGeluC))));
  } else if constexpr (ACT == NVFP4_ACT_SILU) {
    return gate2(z, mul2(z, splat2(-kLog2e)));
  } else if constexpr (sizeof(T) == 4) {
    const float2 d = fma2(splat2(kGaussV), make_float2(fabsf(z.x), fabsf(z.y)), splat2(1.0f));
    const float2 y = mul2(mul2(z, z), splat2(-kHalfLog2e));
    const float2 t = make_float2(rcp(d.x), rcp(d.y)), e = make_float2(ex2(y.x), ex2(y.y));
    float2 q = splat2(gauss_v(8));
#pragma unroll
    for (int i = 7; i >= 0; --i) q = fma2(q, t, splat2(gauss_v(i)));
    q = mul2(mul2(q, t), e);
    const float2 r = sub2(splat2(1.0f), q);
    return mul2(z, make_float2(z.x < 0.0f ? q.x : r.x, z.y < 0.0f ? q.y : r.y));
  } else {
    const float2 x = mul2(make_float2(fabsf(z.x), fabsf(z.y)), splat2(kRsqrt2));
    const float2 d = fma2(splat2(0.3275911f), x, splat2(1.0f)), y = mul2(mul2(splat2(-kLog2e), x), x);
    const float2 t = make_float2(rcp(d.x), rcp(d.y)), e = make_float2(ex2(y.x), ex2(y.y));
    float2 q = fma2(splat2(1.061405429f), t, splat2(-1.453152027f));
    q = fma2(q, t, splat2(1.421413741f));
    q = fma2(q, t, splat2(-0.284496736f));
    q = fma2(q, t, splat2(0.254829592f));
    q = mul2(mul2(mul2(splat2(0.5f), q), t), e);
    const float2 r = sub2(splat2(1.0f), q);
    return mul2(z, make_float2(z.x < 0.0f ? q.x : r.x, z.y < 0.0f ? q.y : r.y));
  }
}
template <int NV, int ACT, typename T>
__device__ __forceinline__ void act_each(float* v) {
#pragma unroll
  for (int i = 0; i < NV; i += 2) {
    const float2 r = act_pair<ACT, T>(make_float2(v[i], v[i + 1]));
    v[i] = r.x;
    v[i + 1] = r.y;
  }
}
// act over a register array, for results of type T; the choice is taken once.
template <int NV, typename T>
__device__ __forceinline__ void act_all(float* v, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: act_each<NV, NVFP4_ACT_RELU, T>(v); break;
    case NVFP4_ACT_GELU: act_each<NV, NVFP4_ACT_GELU, T>(v); break;
    case NVFP4_ACT_GELU_TANH: act_each<NV, NVFP4_ACT_GELU_TANH, T>(v); break;
    case NVFP4_ACT_SILU: act_each<NV, NVFP4_ACT_SILU, T>(v); break;
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
