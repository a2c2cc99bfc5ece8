// linear_split.cu -- nvfp4_linear for few tokens: K split over a cluster.
//
// d = act(alpha_a alpha_b A B^T + bias) + residual where the product is too
// small to fill the GPU with whole output tiles and the weight's bytes (9/16
// per value) are what it costs.  The weight's rows are the MMA's 128 lanes and
// the tokens its BN columns (16 to 128), so that a tile of the weight is
// multiplied once by all tokens.  A cluster of S blocks shares one output tile:
// block r sums its part of K in TMEM, the partial tiles meet in shared memory,
// and each block joins 128 / S features of all S parts (in rank order, so that
// the sum's order is fixed), applies the epilogue and stores.
#include <algorithm>

#include "linear_launch.h"
#include "linear_tc.cuh"

namespace nvfp4 {
namespace lin {
namespace {

constexpr int kThreads = 192;  // warps 0-3: epilogue (TMEM lane quarters), 4: loads, 5: MMA

template <int BN>
struct Cfg {
  static constexpr int kStageBytes = kLaneTile + BN * kBK / 2 + 2 * kSfStage;  // 22 to 36 KB
  static constexpr int kStages = BN == 16 ? 5 : (BN == 32 ? 4 : 3);            // two blocks per SM
  static constexpr int kSmem = kStages * kStageBytes + 256 /* barriers */ + 1024 /* alignment */;
  static constexpr uint32_t kSfCols = 32;  // TMEM columns of one stage's scales
  static constexpr uint32_t kTmemCols = 256;
  static_assert(BN + kStages * kSfCols <= kTmemCols, "TMEM columns (two blocks share 512)");
  static_assert(BN * kLaneRows * 4 <= kStages * kStageBytes, "the partial tile takes the stages' place");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ float ld_rank(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// Epilogue of one output; returns the magnitude bits of the rounded d.
template <typename T>
__device__ __forceinline__ uint32_t put(const LinearArgs& a, int64_t m, int64_t n, float z) {
  if (a.z) static_cast<T*>(a.z)[m * a.ldz + n] = from_f32<T>(z);
  float d = act_value(z, a.act);
  if (a.residual) d += to_f32(static_cast<const T*>(a.residual)[m * a.ldr + n]);
  const T o = from_f32<T>(d);
  static_cast<T*>(a.d)[m * a.ldd + n] = o;
  return abs_bits(to_f32(o));
}

template <int BN, typename T>
__global__ void __launch_bounds__(kThreads)
    linear_split_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap, int S) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t raw[];
  // 1024-byte alignment for the 128-byte swizzle
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::kStages, done = full0 + 16 * C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::kStages + 1);
  volatile int* stop = reinterpret_cast<int*>(bars + 2 * C::kStages + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int64_t f0 = (int64_t)(blockIdx.x / S) * kLaneRows;  // first feature
  const int64_t t0 = (int64_t)blockIdx.y * BN;               // first token
  const Steps K(a.K);
  const int k0 = (int)((int64_t)K.n * rank / S), k1 = (int)((int64_t)K.n * (rank + 1) / S);
  constexpr int kColTile = BN * kBK / 2;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tma::mbar_init(full0 + 8 * s, 1);
      tma::mbar_init(empty0 + 8 * s, 1);
    }
    tma::mbar_init(done, 1);
    *stop = 0;
    tma::fence_barrier_init();
  }
  if (warp == 5) {
    tc5::alloc(smem_u32(tmem_slot), C::kTmemCols);
    tc5::relinquish_alloc_permit();
  }
  tc5::fence_before_thread_sync();
  __syncthreads();
  tc5::fence_after_thread_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    if (lane == 0) {
      const int64_t sf_row = (a.K + 63) / 64 * kSfBlock;  // scale bytes of a 128-row band
      const uint8_t* sfw = a.sfb + f0 / 128 * sf_row;
      const uint8_t* sfx = a.sfa + t0 / 128 * sf_row;
      Ring<C::kStages> r;
      int kb = k0;
      for (; kb < k1; ++kb, r.next()) {
        if (kb - k0 >= C::kStages && !tma::wait(empty0 + 8 * r.slot, r.phase ^ 1u)) {
          *stop = 1;
          break;
        }
        const uint32_t st = smem_u32(smem + r.slot * C::kStageBytes), full = full0 + 8 * r.slot;
        const int groups = K.groups(kb);
        tma::arrive_expect_tx(full, (uint32_t)(kLaneTile + kColTile + 2 * groups * kSfBlock));
        load_codes<BN>(st, full, &wmap, &xmap, (int)f0, (int)t0, kb);
        load_scales(st + kLaneTile + kColTile, full, sfw, sfx, sf_row, kb, groups, 1);
      }
      // no copy may land after the block has gone: wait for the last fill of every stage
      const int g = kb - k0;
      for (int j = g > C::kStages ? g - C::kStages : 0; j < g; ++j)
        tma::wait(full0 + 8 * (j % C::kStages), (uint32_t)(j / C::kStages) & 1u);
    }
  } else if (warp == 5) {
    Ring<C::kStages> r;
    for (int kb = k0; kb < k1; ++kb, r.next()) {
      if (!__all_sync(0xFFFFFFFFu, tma::wait(full0 + 8 * r.slot, r.phase))) {
        if (lane == 0) *stop = 1;
        break;
      }
      const int groups = K.groups(kb);
      uint8_t* st = smem + r.slot * C::kStageBytes;
      if (kb == K.n - 1 && K.tail) clear_tail(st + kLaneTile + kColTile, 2, groups - 1, lane);
      tc5::fence_after_thread_sync();
      if (lane == 0) {
        const uint32_t sf_tmem = tmem + BN + (uint32_t)r.slot * C::kSfCols;
        copy_stage_scales<BN>(sf_tmem, smem_u32(st + kLaneTile + kColTile), groups);
        mma_stage<BN>(tmem, sf_tmem, StageDesc(smem_u32(st)), groups, kb == k0);
        tc5::commit(empty0 + 8 * r.slot);
      }
      __syncwarp();
    }
    if (lane == 0) tc5::commit(done);  // arrives when every MMA issued above has completed
  }
  __syncwarp();

  const bool ready = tma::wait(done, 0);
  const bool ok = __syncthreads_and(ready && *stop == 0);
  tc5::fence_after_thread_sync();
  const float scale = a.alpha_a[0] * a.alpha_b[0];
  const int tokens = (int)(a.M - t0 < BN ? a.M - t0 : BN);
  uint32_t top = 0;
  if (S == 1) {
    if (warp < 4) {
      const int64_t n = f0 + tid;
      const float bias = a.bias && n < a.N ? load_as_f32(a.bias, n, a.bias_bf16) : 0.0f;
#pragma unroll 1
      for (int c = 0; c < BN && c < tokens; c += 16) {
        uint32_t r[16];
        ld_32x32b_x16(tmem + (uint32_t)c + ((uint32_t)(32 * warp) << 16), r);
        tc5::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (ok && n < a.N && c + i < tokens)
            top = max(top, put<T>(a, t0 + c + i, n, fmaf(__uint_as_float(r[i]), scale, bias)));
      }
    }
  } else {
    // the partial tile, one row of 128 features per token, in the stages' place
    float* part = reinterpret_cast<float*>(smem);
    if (warp < 4) {
#pragma unroll 1
      for (int c = 0; c < BN && c < tokens; c += 16) {
        uint32_t r[16];
        ld_32x32b_x16(tmem + (uint32_t)c + ((uint32_t)(32 * warp) << 16), r);
        tc5::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kLaneRows + tid] = __uint_as_float(r[i]);
      }
    }
    cluster_sync();
    const int per = kLaneRows / S;
    const uint32_t base = smem_u32(part);
    for (int i = tid; i < tokens * per; i += kThreads) {
      const int c = i / per, f = (int)rank * per + i % per;
      const int64_t n = f0 + f;
      float v = 0.0f;
      for (int q = 0; q < S; ++q) v += ld_rank(base + 4u * (uint32_t)(c * kLaneRows + f), (uint32_t)q);
      if (ok && n < a.N) {
        const float bias = a.bias ? load_as_f32(a.bias, n, a.bias_bf16) : 0.0f;
        top = max(top, put<T>(a, t0 + c, n, fmaf(v, scale, bias)));
      }
    }
    cluster_sync();  // no block leaves while another reads its part
  }
  if (a.amax) put_amax(a.amax, top);
  if (tid == 0 && !ok && a.status) atomicExch(a.status, kStatusPipeline);
  tc5::fence_before_thread_sync();
  __syncthreads();
  if (warp == 5) tc5::dealloc(tmem, C::kTmemCols);
}

template <int BN, typename T>
cudaError_t launch(const LinearArgs& a, int S, cudaStream_t s) {
  using C = Cfg<BN>;
  auto kern = linear_split_kernel<BN, T>;
  static std::atomic<int> cache[64] = {};
  int cap = 0;
  cudaError_t e = resident_grid(kern, kThreads, C::kSmem, cache, cap);  // opts in to the shared memory
  if (e != cudaSuccess) return e;
  CUtensorMap wmap, xmap;
  e = make_codes_map(&wmap, a.qb, a.N, a.K / 2, kBK / 2, kLaneRows);
  if (e != cudaSuccess) return e;
  e = make_codes_map(&xmap, a.qa, a.M, a.K / 2, kBK / 2, BN);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + kLaneRows - 1) / kLaneRows * S), (unsigned)((a.M + BN - 1) / BN));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, wmap, xmap, S);
}

template <int BN>
cudaError_t launch_t(const LinearArgs& a, int S, cudaStream_t s) {
  return a.out_bf16 ? launch<BN, bf16>(a, S, s) : launch<BN, float>(a, S, s);
}

}  // namespace

cudaError_t launch_split(const LinearArgs& a, int bn, int S, cudaStream_t s) {
  switch (bn) {
    case 16: return launch_t<16>(a, S, s);
    case 32: return launch_t<32>(a, S, s);
    case 64: return launch_t<64>(a, S, s);
    default: return launch_t<128>(a, S, s);
  }
}

}  // namespace lin
}  // namespace nvfp4
