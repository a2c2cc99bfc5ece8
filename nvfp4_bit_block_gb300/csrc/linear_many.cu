// linear_many.cu -- nvfp4_linear for many tokens: persistent blocks walk tiles
// of 128 tokens x BN features.
//
// Warp 0 loads (TMA), warp 1 issues the MMAs, warps 4-7 move each stage's scales
// from shared memory to TMEM (tcgen05.cp from the MMA's thread would run in the
// tensor pipe's order, 12 copies per stage: 970 instead of 645 us for 16384 x 5120
// x 20480), warps 8-15 are the epilogue: two warps per TMEM lane quarter, each
// with half of the tile's columns.  They take the whole accumulator into
// registers and hand it back before they compute, so that the next tile's MMAs
// wait for the read-out alone and the epilogue's arithmetic and traffic run
// beside them; registers are moved to them from the other warps (setmaxnreg).
#include "linear_launch.h"
#include "linear_tc.cuh"

namespace nvfp4 {
namespace lin {
namespace {

constexpr int kThreads = 512;
constexpr int kSfWarp0 = 4, kSfWarps = 4, kEpiWarp0 = 8, kEpiWarps = 8;
// Registers per thread: 512 * 128 at launch, shared out as 256 * 48 + 256 * 208.
constexpr int kFewRegs = 48, kEpiRegs = 208;
static_assert(256 * kFewRegs + 256 * kEpiRegs == kThreads * 128, "register split");
constexpr int64_t kGroupM = 8;  // token tiles walked together, so that blocks in flight share operand tiles in L2

template <int BN>
struct Cfg {
  static constexpr int kBands = BN / 128;
  static constexpr int kSfAt = kLaneTile + BN * kBK / 2;
  static constexpr int kStageBytes = kSfAt + kSfStage * (1 + kBands);  // 54 KB
  static constexpr int kStages = 4;
  static constexpr int kHalf = BN / 2;  // columns of an epilogue warp
  static constexpr int kSmem = kStages * kStageBytes + BN * 4 /* bias */ + 256 /* barriers */ + 1024 /* alignment */;
  static constexpr uint32_t kSfCols = 16 + 16 * kBands;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(BN + kStages * kSfCols <= kTmemCols, "TMEM columns");
  static_assert(kSmem <= 232448, "shared memory");
};

// Named barrier of `threads` threads; true if `v` holds in all of them.
__device__ __forceinline__ bool bar_all(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Tile t -> (token tile, feature tile).
__device__ __forceinline__ void tile_at(int64_t t, int64_t tm, int64_t tn, int64_t& m, int64_t& n) {
  const int64_t per = kGroupM * tn;
  const int64_t g = t / per, r = t - g * per, first = g * kGroupM;
  const int64_t rows = tm - first < kGroupM ? tm - first : kGroupM;
  m = first + r % rows;
  n = r / rows;
}

// 8 consecutive outputs; `p` is 16-byte aligned.
__device__ __forceinline__ void store8(bf16* p, const float* v) {
  uint4 w;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  w.x = *reinterpret_cast<uint32_t*>(&h[0]);
  w.y = *reinterpret_cast<uint32_t*>(&h[1]);
  w.z = *reinterpret_cast<uint32_t*>(&h[2]);
  w.w = *reinterpret_cast<uint32_t*>(&h[3]);
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void add8(const bf16* p, float* v) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  v[0] += bf16_lo(w.x);
  v[1] += bf16_hi(w.x);
  v[2] += bf16_lo(w.y);
  v[3] += bf16_hi(w.y);
  v[4] += bf16_lo(w.z);
  v[5] += bf16_hi(w.z);
  v[6] += bf16_lo(w.w);
  v[7] += bf16_hi(w.w);
}
__device__ __forceinline__ void add8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] += a.x;
  v[1] += a.y;
  v[2] += a.z;
  v[3] += a.w;
  v[4] += b.x;
  v[5] += b.y;
  v[6] += b.z;
  v[7] += b.w;
}

// Epilogue of 32 consecutive features of one token, `v` holding the products.
template <typename T>
__device__ __forceinline__ uint32_t put32(const LinearArgs& a, int64_t m, int64_t n, float* v, const float* bias,
                                          float scale, bool vec) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(bias + i);
    v[i] = fmaf(v[i], scale, b.x);
    v[i + 1] = fmaf(v[i + 1], scale, b.y);
    v[i + 2] = fmaf(v[i + 2], scale, b.z);
    v[i + 3] = fmaf(v[i + 3], scale, b.w);
  }
  uint32_t top = 0;
  if (vec && n + 32 <= a.N) {
    if (a.z) {
      T* p = static_cast<T*>(a.z) + m * a.ldz + n;
#pragma unroll
      for (int i = 0; i < 32; i += 8) store8(p + i, v + i);
    }
    act_all<32>(v, a.act);
    if (a.residual) {
      const T* p = static_cast<const T*>(a.residual) + m * a.ldr + n;
#pragma unroll
      for (int i = 0; i < 32; i += 8) add8(p + i, v + i);
    }
    T* p = static_cast<T*>(a.d) + m * a.ldd + n;
#pragma unroll
    for (int i = 0; i < 32; i += 8) store8(p + i, v + i);
    if (a.amax) {
#pragma unroll
      for (int i = 0; i < 32; ++i) top = max(top, abs_bits(to_f32(from_f32<T>(v[i]))));
    }
  } else {
    const int cols = a.N - n < 32 ? (int)(a.N - n) : 32;
    if (a.z) {
      T* p = static_cast<T*>(a.z) + m * a.ldz + n;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < cols) p[i] = from_f32<T>(v[i]);
    }
    act_all<32>(v, a.act);
    const T* res = a.residual ? static_cast<const T*>(a.residual) + m * a.ldr + n : nullptr;
    T* p = static_cast<T*>(a.d) + m * a.ldd + n;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i < cols) {
        const T o = from_f32<T>(v[i] + (res ? to_f32(res[i]) : 0.0f));
        p[i] = o;
        top = max(top, abs_bits(to_f32(o)));
      }
    }
  }
  return top;
}

template <int BN, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    linear_many_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap xmap,
                       const __grid_constant__ CUtensorMap wmap, int vec) {
  using C = Cfg<BN>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t raw[];
  // 1024-byte alignment for the 128-byte swizzle
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* bias_s = reinterpret_cast<float*>(smem + kStages * C::kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(bias_s + BN);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, sfr0 = empty0 + 8 * kStages;
  const uint32_t accf = sfr0 + 8 * kStages, acce = accf + 8, drain = accf + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + 3);
  volatile int* stop = reinterpret_cast<int*>(bars + 3 * kStages + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Steps K(a.K);
  const int64_t tm = (a.M + kLaneRows - 1) / kLaneRows, tn = (a.N + BN - 1) / BN, tiles = tm * tn;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tma::mbar_init(full0 + 8 * s, 1);
      tma::mbar_init(empty0 + 8 * s, 1);
      tma::mbar_init(sfr0 + 8 * s, kSfWarps);  // the stage has arrived and its scales are in TMEM
    }
    tma::mbar_init(accf, 1);
    tma::mbar_init(acce, kEpiWarps);
    tma::mbar_init(drain, 1);
    *stop = 0;
    tma::fence_barrier_init();
  }
  if (warp == 1) {
    tc5::alloc(smem_u32(tmem_slot), C::kTmemCols);
    tc5::relinquish_alloc_permit();
  }
  tc5::fence_before_thread_sync();
  __syncthreads();
  tc5::fence_after_thread_sync();
  const uint32_t tmem = *tmem_slot;
  uint32_t top = 0;

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
      if (lane == 0) {
        const int64_t sf_row = (a.K + 63) / 64 * kSfBlock;  // scale bytes of a 128-row band
        Ring<kStages> r;
        int64_t g = 0;
        for (int64_t t = blockIdx.x; t < tiles && !*stop; t += gridDim.x) {
          int64_t m, n;
          tile_at(t, tm, tn, m, n);
          const int bands = a.N - n * BN > 128 ? C::kBands : 1;  // 128-row bands of scales that exist
          const uint8_t* sfx = a.sfa + m * sf_row;
          const uint8_t* sfw = a.sfb + n * C::kBands * sf_row;
          for (int kb = 0; kb < K.n; ++kb, ++g, r.next()) {
            if (g >= kStages && !tma::wait(empty0 + 8 * r.slot, r.phase ^ 1u)) {
              *stop = 1;
              break;
            }
            const uint32_t st = smem_u32(smem + r.slot * C::kStageBytes), full = full0 + 8 * r.slot;
            const int groups = K.groups(kb);
            tma::arrive_expect_tx(full, (uint32_t)(C::kSfAt + (1 + bands) * groups * kSfBlock));
            load_codes<BN>(st, full, &xmap, &wmap, (int)(m * kLaneRows), (int)(n * BN), kb);
            load_scales(st + C::kSfAt, full, sfx, sfw, sf_row, kb, groups, bands);
          }
        }
        // no copy may land after the block has gone: wait for the last fill of every stage
        for (int64_t j = g > kStages ? g - kStages : 0; j < g; ++j)
          tma::wait(full0 + 8 * (int)(j % kStages), (uint32_t)(j / kStages) & 1u);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        Ring<kStages> r;
        int li = 0;
        for (int64_t t = blockIdx.x; t < tiles && !*stop; t += gridDim.x, ++li) {
          // the epilogue has taken the previous tile out
          if (li > 0 && !tma::wait(acce, (uint32_t)(li - 1) & 1u)) {
            *stop = 1;
            break;
          }
          for (int kb = 0; kb < K.n; ++kb, r.next()) {
            if (!tma::wait(sfr0 + 8 * r.slot, r.phase)) {  // the scale warps have waited for the stage
              *stop = 1;
              break;
            }
            tc5::fence_after_thread_sync();
            mma_stage<BN>(tmem, tmem + BN + (uint32_t)r.slot * C::kSfCols,
                          StageDesc(smem_u32(smem + r.slot * C::kStageBytes)), K.groups(kb), kb == 0);
            tc5::commit(empty0 + 8 * r.slot);
          }
          if (*stop) break;
          tc5::commit(accf);
        }
        tc5::commit(drain);  // arrives when every MMA issued above has completed
      }
    } else if (warp >= kSfWarp0) {
      const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
      Ring<kStages> r;
      bool quit = false;
      for (int64_t t = blockIdx.x; t < tiles && !quit; t += gridDim.x) {
        for (int kb = 0; kb < K.n; ++kb, r.next()) {
          quit = !__all_sync(0xFFFFFFFFu, tma::wait(full0 + 8 * r.slot, r.phase) && *stop == 0);
          if (quit) break;
          put_scales<C::kBands>(tmem + quarter + BN + (uint32_t)r.slot * C::kSfCols,
                                smem + r.slot * C::kStageBytes + C::kSfAt, K.groups(kb), kb == K.n - 1 && K.tail, lane);
          tc5::fence_before_thread_sync();
          __syncwarp();
          if (lane == 0) arrive(sfr0 + 8 * r.slot);
        }
      }
      if (quit && lane == 0) *stop = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int e = warp - kEpiWarp0, q = warp & 3, half = e >> 2;  // lane quarter, column half
    const float scale = a.alpha_a[0] * a.alpha_b[0];
    float* bias = bias_s + half * C::kHalf;  // shared by the half's four warps
    int li = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++li) {
      int64_t m, n;
      tile_at(t, tm, tn, m, n);
      const int64_t row = m * kLaneRows + 32 * q + lane, col = n * BN + half * C::kHalf;
      // the four warps of this half have read the previous tile's bias; load this tile's
      bar_all(1 + half, 128, true);
      for (int i = 32 * q + lane; i < C::kHalf; i += 128)
        bias[i] = a.bias && col + i < a.N ? load_as_f32(a.bias, col + i, a.bias_bf16) : 0.0f;
      const bool ready = tma::wait(accf, (uint32_t)li & 1u);
      // the barrier orders the bias, and the four warps go on or stop together
      if (!bar_all(1 + half, 128, ready && *stop == 0)) {
        if (lane == 0) *stop = 1;
        break;
      }
      tc5::fence_after_thread_sync();
      const uint32_t acc = tmem + (uint32_t)(half * C::kHalf) + ((uint32_t)(32 * q) << 16);
      uint32_t r[C::kHalf];
#pragma unroll
      for (int c = 0; c < C::kHalf; c += 32) tc5::ld_32x32b_x32(acc + (uint32_t)c, r + c);
      tc5::wait_ld();
      tc5::fence_before_thread_sync();
      __syncwarp();
      if (lane == 0) arrive(acce);
      if (row < a.M) {
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 32)
          if (col + c < a.N)
            top = max(top, put32<T>(a, row, col + c, reinterpret_cast<float*>(r + c), bias + c, scale, vec != 0));
      }
    }
  }
  __syncwarp();
  __syncthreads();
  const bool drained = tma::wait(drain, 0);
  if (a.amax && warp >= kEpiWarp0) put_amax(a.amax, top);
  if (tid == 0 && (*stop || !drained) && a.status) atomicExch(a.status, kStatusPipeline);
  tc5::fence_before_thread_sync();
  __syncthreads();
  if (warp == 1) tc5::dealloc(tmem, C::kTmemCols);
}

template <int BN, typename T>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
  using C = Cfg<BN>;
  auto kern = linear_many_kernel<BN, T>;
  static std::atomic<int> cache[64] = {};
  int cap = 0;
  cudaError_t e = resident_grid(kern, kThreads, C::kSmem, cache, cap);
  if (e != cudaSuccess) return e;
  CUtensorMap xmap, wmap;
  e = make_codes_map(&xmap, a.qa, a.M, a.K / 2, kBK / 2, kLaneRows);
  if (e != cudaSuccess) return e;
  e = make_codes_map(&wmap, a.qb, a.N, a.K / 2, kBK / 2, BN);
  if (e != cudaSuccess) return e;
  auto ok16 = [](const void* p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0);
  };
  const int vec = ok16(a.d, a.ldd) && ok16(a.z, a.ldz) && ok16(a.residual, a.ldr);
  const int64_t tiles = ((a.M + kLaneRows - 1) / kLaneRows) * ((a.N + BN - 1) / BN);
  kern<<<(unsigned)(tiles < cap ? tiles : cap), kThreads, C::kSmem, s>>>(a, xmap, wmap, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_many(const LinearArgs& a, cudaStream_t s) {
  return a.out_bf16 ? launch<256, bf16>(a, s) : launch<256, float>(a, s);
}

}  // namespace lin
}  // namespace nvfp4
