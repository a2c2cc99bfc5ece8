// linear_many.cu -- nvfp4_linear for many tokens: pairs of blocks walk tiles of
// 256 tokens x 256 features.
//
// What bounds the product is the rate at which an SM takes operands from L2 (64
// bytes per clock): a stage of 256 values of K feeds 512 clocks of MMAs, and a
// block on its own with a 128 x 256 tile needs 54 KB for it.  In a pair
// (cta_group::2) each block holds its 128 tokens and half of the weight's rows,
// 38 KB: 256 x 256 outputs from the bytes of two 128 x 128 tiles.
//
// In each block: warp 0 loads its part of a stage (TMA); warps 4-7 wait for the
// stage, move its scales from shared memory to TMEM (tcgen05.cp from the MMA's
// thread would run in the tensor pipe's order, 12 copies per stage: 970 instead
// of 650 us for 16384 x 5120 x 20480) and tell the leader block, whose warp 1
// issues the pair's MMAs.  Warps 8-15 are the epilogue: two warps per TMEM lane
// quarter, each with half of the tile's columns.  They take the whole
// accumulator into registers and hand it back before they compute, so that the
// next tile's MMAs wait for the read-out alone; registers are moved to them
// from the other warps (setmaxnreg).  Outputs are staged in shared memory, 32
// rows of 64 bytes per warp, and stored by TMA as whole sectors (16-byte pieces
// of 32 rows at once cost 3 us per tile); the residual comes in by TMA before the
// product is done.
#include "linear_launch.h"
#include "linear_tc.cuh"

namespace nvfp4 {
namespace lin {
namespace {

constexpr int kBN = 256;
constexpr int kThreads = 512;
constexpr int kSfWarp0 = 4, kSfWarps = 4, kEpiWarp0 = 8, kEpiWarps = 8;
// Registers per thread: 512 * 128 at launch, shared out as 256 * 48 + 256 * 208.
constexpr int kFewRegs = 48, kEpiRegs = 208;
static_assert(256 * kFewRegs + 256 * kEpiRegs == kThreads * 128, "register split");
constexpr int64_t kGroupM = 8;  // token tiles walked together, so that blocks in flight share operand tiles in L2

constexpr int kBands = 2;                                    // 128-row scale bands of the features
constexpr int kSfAt = 2 * kLaneTile;                         // codes of 128 tokens and 128 features
constexpr int kStageBytes = kSfAt + kSfStage * (1 + kBands);  // 38 KB
constexpr int kStages = 5;
constexpr int kHalf = kBN / 2;  // columns of an epilogue warp
constexpr int kRow = 64;         // staging buffers: 32 rows of 64 bytes, two per epilogue warp
constexpr int kBox = 32 * kRow;
constexpr int kStageOut = kEpiWarps * 2 * kBox;
constexpr int kBars = 3 * kStages + 3 + 2 * kEpiWarps;
constexpr int kSmem = kStages * kStageBytes + kStageOut + kBN * 4 /* bias */ + 512 /* barriers */ + 1024 /* alignment */;
constexpr uint32_t kSfCols = 16 + 16 * kBands;
constexpr uint32_t kTmemCols = 512;
static_assert(kBN + kStages * kSfCols <= kTmemCols, "TMEM columns");
static_assert(2 * kBox == 32 * 32 * 4, "a warp's staging buffers hold a square of 32 x 32 values");
static_assert(kStageBytes % 1024 == 0 && 8 * (kBars + 2) <= 512 && kSmem <= 232448, "shared memory");

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

// 16 bytes of outputs: 8 bf16 or 4 fp32 values, rounded.
__device__ __forceinline__ uint4 pack16(const float* v, bf16) {
  uint4 w;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  w.x = *reinterpret_cast<uint32_t*>(&h[0]);
  w.y = *reinterpret_cast<uint32_t*>(&h[1]);
  w.z = *reinterpret_cast<uint32_t*>(&h[2]);
  w.w = *reinterpret_cast<uint32_t*>(&h[3]);
  return w;
}
__device__ __forceinline__ uint4 pack16(const float* v, float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void add16(uint4 w, float* v, bf16) {
  v[0] += bf16_lo(w.x);
  v[1] += bf16_hi(w.x);
  v[2] += bf16_lo(w.y);
  v[3] += bf16_hi(w.y);
  v[4] += bf16_lo(w.z);
  v[5] += bf16_hi(w.z);
  v[6] += bf16_lo(w.w);
  v[7] += bf16_hi(w.w);
}
__device__ __forceinline__ void add16(uint4 w, float* v, float) {
  v[0] += __uint_as_float(w.x);
  v[1] += __uint_as_float(w.y);
  v[2] += __uint_as_float(w.z);
  v[3] += __uint_as_float(w.w);
}

// Largest magnitude among 16 bytes of outputs, joined to `top` (NaN is the largest).
__device__ __forceinline__ uint32_t top16(uint4 w, uint32_t top, bf16) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w.x), "r"(w.y));
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w.z));
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w.w));
  m &= 0x7FFF7FFFu;
  return max(top, max(m << 16, m & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t top16(uint4 w, uint32_t top, float) {
  const uint32_t k = 0x7FFFFFFFu;
  return max(max(top, max(w.x & k, w.y & k)), max(w.z & k, w.w & k));
}

// v = product * scale + bias.
template <int NV>
__device__ __forceinline__ void affine(float* v, const float* bias, float scale) {
#pragma unroll
  for (int i = 0; i < NV; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(bias + i);
    const float2 lo = fma2(make_float2(v[i], v[i + 1]), splat2(scale), make_float2(b.x, b.y));
    const float2 hi = fma2(make_float2(v[i + 2], v[i + 3]), splat2(scale), make_float2(b.z, b.w));
    v[i] = lo.x;
    v[i + 1] = lo.y;
    v[i + 2] = hi.x;
    v[i + 3] = hi.y;
  }
}

// Outputs that cannot go through a tensor map (rows that do not begin and end at 16
// bytes), or a z beside a residual: 32 rows x 32 features of a warp.  `v` is this lane's
// row of products; through `tile` (32 x 32 values, element (r, c) at column c ^ r, so
// that neither its rows nor its columns meet in a bank) the lanes become columns
// and each access to memory is a piece of one row, 16 rows at a time (4096 x 20479
// x 5120: 202 us; with a row per lane and scalar accesses 798 us).
template <typename T, bool FULL>
__device__ __forceinline__ uint32_t put_rows(const LinearArgs& a, T* d, T* z, const T* res, const float* tile, int rows,
                                             float bias, float scale, uint32_t top) {
  const int lane = threadIdx.x & 31;
  constexpr int B = 16;  // rows at a time
#pragma unroll 1
  for (int r0 = 0; r0 < 32 && (FULL || r0 < rows); r0 += B) {
    float w[B];
    T add[B];
    if (res) {
#pragma unroll
      for (int i = 0; i < B; ++i, res += a.ldr) add[i] = FULL || r0 + i < rows ? *res : from_f32<T>(0.0f);
    }
    const int x = lane ^ r0;  // B divides r0: lane ^ (r0 + i) = x ^ i
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = fmaf(tile[(r0 + i) * 32 + (x ^ i)], scale, bias);
    if (z) {
#pragma unroll
      for (int i = 0; i < B; ++i, z += a.ldz)
        if (FULL || r0 + i < rows) *z = from_f32<T>(w[i]);
    }
    act_all<B, T>(w, a.act);
    if (res) {
#pragma unroll
      for (int i = 0; i < B; ++i) w[i] += to_f32(add[i]);
    }
#pragma unroll
    for (int i = 0; i < B; ++i, d += a.ldd) {
      if (FULL || r0 + i < rows) {
        const T o = from_f32<T>(w[i]);
        *d = o;
        top = max(top, abs_bits(to_f32(o)));
      }
    }
  }
  return top;
}
template <typename T>
__device__ __forceinline__ uint32_t put_square(const LinearArgs& a, int64_t row0, int64_t n, const float* v, float* tile,
                                               float bias, float scale, uint32_t top) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 32; ++c) tile[lane * 32 + (c ^ lane)] = v[c];
  __syncwarp();
  const int rows = a.M - row0 < 32 ? (int)(a.M - row0) : 32;
  if (n + lane < a.N) {
    T* d = static_cast<T*>(a.d) + row0 * a.ldd + n + lane;
    T* z = a.z ? static_cast<T*>(a.z) + row0 * a.ldz + n + lane : nullptr;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + row0 * a.ldr + n + lane : nullptr;
    top = rows == 32 ? put_rows<T, true>(a, d, z, res, tile, rows, bias, scale, top)
                     : put_rows<T, false>(a, d, z, res, tile, rows, bias, scale, top);
  }
  __syncwarp();
  return top;
}

// This lane's row of a staging buffer in the 64-byte swizzle: 16-byte piece i.
__device__ __forceinline__ uint4* piece(uint8_t* buf, int lane, int i) {
  return reinterpret_cast<uint4*>(buf + lane * kRow + ((i ^ ((lane >> 1) & 3)) << 4));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    linear_many_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap xmap,
                       const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap dmap,
                       const __grid_constant__ CUtensorMap zmap, const __grid_constant__ CUtensorMap rmap, int staged) {
  extern __shared__ uint8_t raw[];
  // 1024-byte alignment for the 128-byte swizzle
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_s = smem + kStages * kStageBytes;
  float* bias_s = reinterpret_cast<float*>(out_s + kStageOut);
  uint64_t* bars = reinterpret_cast<uint64_t*>(bias_s + kBN);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, sfr0 = empty0 + 8 * kStages;
  const uint32_t accf = sfr0 + 8 * kStages, acce = accf + 8, drain = accf + 16, res0 = accf + 24;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* stop = reinterpret_cast<int*>(bars + kBars + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();  // 0: the leader
  const Steps K(a.K);
  const int64_t tm = (a.M + 2 * kLaneRows - 1) / (2 * kLaneRows), tn = (a.N + kBN - 1) / kBN, tiles = tm * tn;
  const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tma::mbar_init(full0 + 8 * s, 1);
      tma::mbar_init(empty0 + 8 * s, 1);
      tma::mbar_init(sfr0 + 8 * s, 2 * kSfWarps);  // leader's: the stage is there in both blocks, its scales in TMEM
    }
    tma::mbar_init(accf, 1);
    tma::mbar_init(acce, 2 * kEpiWarps);  // leader's: both blocks have taken the tile out
    tma::mbar_init(drain, 1);
    for (int i = 0; i < 2 * kEpiWarps; ++i) tma::mbar_init(res0 + 8 * i, 1);
    *stop = 0;
    tma::fence_barrier_init();
  }
  if (warp == 1) {
    alloc2(smem_u32(tmem_slot), kTmemCols);
    relinquish2();
  }
  tc5::fence_before_thread_sync();
  __syncthreads();
  cluster_sync();  // both blocks' barriers are set up
  tc5::fence_after_thread_sync();
  // what came before may run beside the setup; from here on memory is read and written
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  uint32_t top = 0;

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
      if (lane == 0) {
        const int64_t sf_row = (a.K + 63) / 64 * kSfBlock;  // scale bytes of a 128-row band
        Ring<kStages> r;
        int64_t g = 0;
        for (int64_t t = first; t < tiles && !*stop; t += step) {
          int64_t m, n;
          tile_at(t, tm, tn, m, n);
          const int64_t row = (2 * m + rank) * kLaneRows, col = n * kBN + rank * kLaneRows;
          const int bands = a.N - n * kBN > 128 ? 2 : 1;  // 128-row bands of scales that exist
          const int tok = row < a.M ? 1 : 0;              // and of the tokens'
          const uint8_t* sfx = a.sfa + (2 * m + rank) * sf_row;
          const uint8_t* sfw = a.sfb + n * kBands * sf_row;
          for (int kb = 0; kb < K.n; ++kb, ++g, r.next()) {
            if (g >= kStages && !tma::wait(empty0 + 8 * r.slot, r.phase ^ 1u)) {
              *stop = 1;
              break;
            }
            const uint32_t st = smem_u32(smem + r.slot * kStageBytes), full = full0 + 8 * r.slot;
            const uint32_t bytes = (uint32_t)(K.groups(kb) * kSfBlock);
            tma::arrive_expect_tx(full, (uint32_t)kSfAt + bytes * (uint32_t)(tok + bands));
            if (!kCopies) continue;
            load_codes(st, full, &xmap, &wmap, (int)row, (int)col, kb);
            const int64_t at = (int64_t)kb * kSfStage;
            if (tok) tc5::bulk_g2s(st + kSfAt, sfx + at, bytes, full);
            tc5::bulk_g2s(st + kSfAt + kSfStage, sfw + at, bytes, full);
            if (bands == 2) tc5::bulk_g2s(st + kSfAt + 2 * kSfStage, sfw + sf_row + at, bytes, full);
          }
        }
        // no copy may land after the block has gone: wait for the last fill of every stage
        for (int64_t j = g > kStages ? g - kStages : 0; j < g && kCopies; ++j)
          tma::wait(full0 + 8 * (int)(j % kStages), (uint32_t)(j / kStages) & 1u);
      }
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        Ring<kStages> r;
        int li = 0;
        for (int64_t t = first; t < tiles && !*stop; t += step, ++li) {
          // both epilogues have taken the previous tile out
          if (li > 0 && !wait_cluster(acce, (uint32_t)(li - 1) & 1u)) {
            *stop = 1;
            break;
          }
          for (int kb = 0; kb < K.n; ++kb, r.next()) {
            if (!wait_cluster(sfr0 + 8 * r.slot, r.phase)) {  // the scale warps have waited for the stage
              *stop = 1;
              break;
            }
            tc5::fence_after_thread_sync();
            mma2_stage<kBN>(tmem, tmem + kBN + (uint32_t)r.slot * kSfCols, StageDesc(smem_u32(smem + r.slot * kStageBytes)),
                            K.groups(kb), kb == 0);
            commit2(empty0 + 8 * r.slot);
          }
          if (*stop) break;
          commit2(accf);
        }
        commit2(drain);  // arrives in both blocks when every MMA issued above has completed
      }
    } else if (warp >= kSfWarp0) {
      const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
      Ring<kStages> r;
      bool quit = false;
      for (int64_t t = first; t < tiles && !quit; t += step) {
        for (int kb = 0; kb < K.n; ++kb, r.next()) {
          quit = !__all_sync(0xFFFFFFFFu, tma::wait(full0 + 8 * r.slot, r.phase) && *stop == 0);
          if (quit) break;
          put_scales<kBands>(tmem + quarter + kBN + (uint32_t)r.slot * kSfCols, smem + r.slot * kStageBytes + kSfAt,
                             K.groups(kb), kb == K.n - 1 && K.tail, lane);
          tc5::fence_before_thread_sync();
          __syncwarp();
          if (lane == 0) arrive_at(sfr0 + 8 * r.slot, 0);
        }
      }
      if (quit && lane == 0) *stop = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    constexpr int kCols = kRow / (int)sizeof(T);   // columns of a staging buffer
    constexpr int kChunks = kHalf / kCols;
    constexpr int kPer = 16 / (int)sizeof(T);    // values in 16 bytes
    const int e = warp - kEpiWarp0, q = warp & 3, half = e >> 2;  // lane quarter, column half
    const float scale = a.alpha_a[0] * a.alpha_b[0];
    float* bias = bias_s + half * kHalf;  // shared by the half's four warps
    uint8_t* buf = out_s + e * 2 * kBox;
    const uint32_t res = res0 + 16 * e;
    int li = 0, slot = 0;
    uint32_t res_phase = 0;
    for (int64_t t = first; t < tiles; t += step, ++li) {
      int64_t m, n;
      tile_at(t, tm, tn, m, n);
      const int64_t row0 = (2 * m + rank) * kLaneRows + 32 * q, row = row0 + lane, col = n * kBN + half * kHalf;
      const bool rows = row0 < a.M;  // warp-uniform: some row of this warp exists
      auto load_res = [&](int c) {   // the residual of chunk c into its buffer, once earlier stores have left it
        if (lane == 0 && rows && col + c * kCols < a.N) {
          stores_read<0>();
          tma::arrive_expect_tx(res + 8 * (c & 1), kBox);
          tma::load_2d(smem_u32(buf + (c & 1) * kBox), &rmap, (int)(col + c * kCols), (int)row0, res + 8 * (c & 1));
        }
      };
      if (staged && a.residual) {
        load_res(0);
        load_res(1);
      }
      // the four warps of this half have read the previous tile's bias; load this tile's
      bar_all(1 + half, 128, true);
      for (int i = 32 * q + lane; i < kHalf; i += 128)
        bias[i] = a.bias && col + i < a.N ? load_as_f32(a.bias, col + i, a.bias_bf16) : 0.0f;
      const bool ready = tma::wait(accf, (uint32_t)li & 1u);
      // the barrier orders the bias, and the four warps go on or stop together
      if (!bar_all(1 + half, 128, ready && *stop == 0)) {
        if (lane == 0) *stop = 1;
        if (staged && a.residual && rows)  // the copies issued above land before the block goes
          for (int c = 0; c < 2 && col + c * kCols < a.N; ++c) tma::wait(res + 8 * c, (res_phase >> c) & 1u);
        break;
      }
      tc5::fence_after_thread_sync();
      const uint32_t acc = tmem + (uint32_t)(half * kHalf) + ((uint32_t)(32 * q) << 16);
      uint32_t raw_r[kHalf];
      float* r = reinterpret_cast<float*>(raw_r);
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) tc5::ld_32x32b_x32(acc + (uint32_t)c, raw_r + c);
      tc5::wait_ld();
      tc5::fence_before_thread_sync();
      __syncwarp();
      if (lane == 0) arrive_at(acce, 0);
      if (!rows) continue;
      if (staged) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (col + c * kCols >= a.N) break;
          float* v = r + c * kCols;
          affine<kCols>(v, bias + c * kCols, scale);
          uint32_t most = 0;
          auto put = [&](const CUtensorMap* map, uint8_t* b) {  // v, rounded, through buffer b
#pragma unroll
            for (int i = 0; i < kRow / 16; ++i) {
              const uint4 w = pack16(v + i * kPer, T());
              *piece(b, lane, i) = w;
              most = top16(w, i == 0 ? 0u : most, T());
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) store_2d(map, (int)(col + c * kCols), (int)row0, smem_u32(b));
          };
          auto next_buffer = [&]() {  // the buffer of two stores ago
            if (lane == 0) stores_read<1>();
            __syncwarp();
            slot ^= 1;
            return buf + slot * kBox;
          };
          if (a.z) put(&zmap, next_buffer());
          act_all<kCols, T>(v, a.act);
          if (a.residual) {
            uint8_t* b = buf + (c & 1) * kBox;
            const uint32_t bit = 1u << (c & 1);
            if (!__all_sync(0xFFFFFFFFu, tma::wait(res + 8 * (c & 1), (res_phase & bit) ? 1u : 0u)) && lane == 0) *stop = 1;
            res_phase ^= bit;
#pragma unroll
            for (int i = 0; i < kRow / 16; ++i) add16(*piece(b, lane, i), v + i * kPer, T());
            put(&dmap, b);
            if (c + 2 < kChunks) load_res(c + 2);
          } else {
            put(&dmap, next_buffer());
          }
          if (a.amax && row < a.M) {
            const int64_t left = a.N - col - c * kCols;
            if (left < kCols) {  // only these are outputs
              most = 0;
#pragma unroll
              for (int i = 0; i < kCols; ++i)
                if (i < left) most = max(most, abs_bits(to_f32(from_f32<T>(v[i]))));
            }
            top = max(top, most);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < kHalf; c += 32)
          if (col + c < a.N) top = put_square<T>(a, row0, col + c, r + c, reinterpret_cast<float*>(buf), bias[c + lane], scale, top);
      }
    }
    if (lane == 0) stores_done();
  }
  __syncwarp();
  __syncthreads();
  const bool drained = tma::wait(drain, 0);
  if (a.amax && warp >= kEpiWarp0) put_amax(a.amax, top);
  if (tid == 0 && (*stop || !drained) && a.status) atomicExch(a.status, kStatusPipeline);
  tc5::fence_before_thread_sync();
  __syncthreads();
  cluster_sync();  // neither block leaves while the pair's MMAs may read it or its peer arrives on its barriers
  if (warp == 1) dealloc2(tmem, kTmemCols);
}

template <typename T>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
  auto kern = linear_many_kernel<T>;
  static std::atomic<int> cache[64] = {};
  int cap = 0;
  cudaError_t e = resident_grid(kern, kThreads, kSmem, cache, cap);
  if (e != cudaSuccess) return e;
  auto ok16 = [](const void* p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0);
  };
  // A TMA store writes a row's last 16 bytes whole, so rows that end inside them would lose what lies behind them.
  // (Leaving only that piece to plain stores took the other products with it: 16384 x 20480 x 5120 with everything on
  // 741 -> 752 us, in fp32 711 -> 732.)
  const bool staged = a.N * (int64_t)sizeof(T) % 16 == 0 && ok16(a.d, a.ldd) && ok16(a.z, a.ldz) &&
                      ok16(a.residual, a.ldr) && !(a.z && a.residual);
  CUtensorMap xmap, wmap, dmap, zmap, rmap;
  e = make_codes_map(&xmap, a.qa, a.M, a.K / 2, kBK / 2, kLaneRows);
  if (e == cudaSuccess) e = make_codes_map(&wmap, a.qb, a.N, a.K / 2, kBK / 2, kLaneRows);
  const bool b16 = sizeof(T) == 2;
  if (e == cudaSuccess) e = make_out_map(&dmap, staged ? a.d : nullptr, b16, a.M, a.N, a.ldd, 32);
  if (e == cudaSuccess) e = make_out_map(&zmap, staged ? a.z : nullptr, b16, a.M, a.N, a.ldz, 32);
  if (e == cudaSuccess) e = make_out_map(&rmap, staged ? a.residual : nullptr, b16, a.M, a.N, a.ldr, 32);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((a.M + 255) / 256) * ((a.N + kBN - 1) / kBN);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (tiles < cap / 2 ? tiles : cap / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, xmap, wmap, dmap, zmap, rmap, staged ? 1 : 0);
}

}  // namespace

cudaError_t launch_many(const LinearArgs& a, cudaStream_t s) {
  return a.out_bf16 ? launch<bf16>(a, s) : launch<float>(a, s);
}

}  // namespace lin
}  // namespace nvfp4
