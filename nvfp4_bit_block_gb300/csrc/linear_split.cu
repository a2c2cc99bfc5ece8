// linear_split.cu -- nvfp4_linear for few tokens: the weight streamed once, K
// split over the SMs.
//
// d = act(alpha_a alpha_b A B^T + bias) + residual where there are too few whole
// output tiles to fill the GPU and the weight's bytes (9/16 per value) are what
// it costs.  The weight's rows are the MMA's 128 lanes and the tokens its BN
// columns (16 to 128), so that a tile of the weight is read once for all tokens.
// The steps of K (256 values) of all output tiles form one row of work that is cut
// into equal pieces, one per SM: every SM streams the same number of bytes,
// without a pause at the tiles' borders, with a ring of stages as deep as shared
// memory holds (200 KB on its way per SM).  A piece leaves the sums of each tile
// that it touches (usually two) in the workspace, and a second, small kernel adds
// the pieces of a tile in order and applies the epilogue; it is launched early
// and waits for the first.  Where the product is so small that whole tiles take
// an SM no longer than that second kernel does, the cuts are between tiles, the
// first kernel applies the epilogue and there is no second.
#include <algorithm>
#include <type_traits>

#include "linear_launch.h"
#include "linear_tc.cuh"

namespace nvfp4 {
namespace lin {
namespace {

// Warps 0-3: sums out of TMEM (its lane quarters), 4-7: scales into TMEM (by
// tensor-core copies from the MMA's thread a stage took twice its bytes' time), 8: loads, 9: MMA.
constexpr int kThreads = 320;
constexpr int kSfWarp0 = 4, kSfWarps = 4, kLoadWarp = 8, kMmaWarp = 9;

template <int BN>
struct Cfg {
  static constexpr int kColTile = BN * kBK / 2;
  static constexpr int kSfAt = kLaneTile + kColTile;
  static constexpr int kStageBytes = kSfAt + 2 * kSfStage;  // 22 to 36 KB
  static constexpr int kStages = BN == 16 ? 10 : (BN == 32 ? 9 : (BN == 64 ? 8 : 6));
  static constexpr int kBars = 3 * kStages + 5;
  static constexpr int kSmem = kStages * kStageBytes + 512 /* barriers */ + 1024 /* alignment */;
  static constexpr uint32_t kSfCols = 32;  // TMEM columns of one stage's scales
  static constexpr uint32_t kTmemCols = 512;
  static_assert(2 * BN + kStages * kSfCols <= kTmemCols, "TMEM columns");
  static_assert(8 * (kBars + 2) <= 512 && kSmem <= 232448, "shared memory");
};

// The work in steps of K: `steps` per output tile, `tiles` of them, cut into `pieces`;
// piece p begins at step floor(tiles * steps * p / pieces), or with whole tiles
// at tile floor(tiles * p / pieces).
struct Cut {
  int64_t tiles, tiles_f;   // output tiles; of them per token tile
  int steps, pieces, most;  // most: pieces that touch a tile at most
  int whole;                // cuts between tiles only
  __host__ __device__ int64_t begin(int64_t piece) const {
    return whole ? tiles * piece / pieces * steps : tiles * steps * piece / pieces;
  }
  // The piece that holds this step: the last p with begin(p) <= step.
  __device__ int piece_of(int64_t step) const {
    const uint64_t n = (uint64_t)(step + 1) * (uint32_t)pieces - 1, d = (uint64_t)tiles * (uint32_t)steps;
    return n >> 32 ? (int)(n / d) : (int)((uint32_t)n / (uint32_t)d);
  }
};

// Epilogue of feature n of `count` (at most 16) tokens from m on, `v` holding the products.
template <typename T>
__device__ __forceinline__ void put_tokens(const LinearArgs& a, int64_t m, int64_t n, int count, float* v, float scale,
                                           float bias) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], scale, bias);
  if (a.z) {
    T* z = static_cast<T*>(a.z) + m * a.ldz + n;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < count) z[i * a.ldz] = from_f32<T>(v[i]);
  }
  act_all<16, T>(v, a.act);
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + m * a.ldr + n;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < count) v[i] += to_f32(r[i * a.ldr]);
  }
  T* d = static_cast<T*>(a.d) + m * a.ldd + n;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < count) d[i * a.ldd] = from_f32<T>(v[i]);
}

// T: type of d where the tiles are whole; void where their sums go to the workspace.
template <int BN, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    linear_split_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap, const Cut cut) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t raw[];
  // 1024-byte alignment for the 128-byte swizzle
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::kStages;
  const uint32_t sfr0 = empty0 + 8 * C::kStages;
  const uint32_t accf0 = sfr0 + 8 * C::kStages, acce0 = accf0 + 16, drain = accf0 + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* stop = reinterpret_cast<int*>(bars + C::kBars + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Steps K(a.K);
  const int64_t u0 = cut.begin(blockIdx.x), u1 = cut.begin((int64_t)blockIdx.x + 1);

  // The loads of this piece, continued by the loading thread from where it left off.
  int64_t u = u0, f = u0 / K.n, tok = f / cut.tiles_f;
  int kb = (int)(u0 - f * K.n);
  f -= tok * cut.tiles_f;
  Ring<C::kStages> fill;
  const int64_t sf_row = (a.K + 63) / 64 * kSfBlock;  // scale bytes of a 128-row band
  auto load_next = [&]() {
    const uint32_t st = smem_u32(smem + fill.slot * C::kStageBytes), full = full0 + 8 * fill.slot;
    const int groups = K.groups(kb);
    tma::arrive_expect_tx(full, (uint32_t)(C::kSfAt + 2 * groups * kSfBlock));
    load_codes(st, full, &wmap, &xmap, (int)(f * kLaneRows), (int)(tok * BN), kb);
    load_scales(st + C::kSfAt, full, a.sfb + f * sf_row, a.sfa + tok * BN / 128 * sf_row, sf_row, kb, groups, 1);
    if (++kb == K.n) {
      kb = 0;
      if (++f == cut.tiles_f) {
        f = 0;
        ++tok;
      }
    }
    ++u;
    fill.next();
  };

  // The setup may run beside the end of the kernel before this one; from griddepcontrol.wait on memory is read and
  // written, and the second kernel may start its own setup.  The first two stages are on their way before the rest of
  // the block is ready (more would keep it waiting).
  if (warp == kLoadWarp && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tma::mbar_init(full0 + 8 * s, 1);
      tma::mbar_init(empty0 + 8 * s, 1);
      tma::mbar_init(sfr0 + 8 * s, kSfWarps);  // the stage has arrived and its scales are in TMEM
    }
    for (int b = 0; b < 2; ++b) {
      tma::mbar_init(accf0 + 8 * b, 1);
      tma::mbar_init(acce0 + 8 * b, 4);
    }
    tma::mbar_init(drain, 1);
    *stop = 0;
    tma::fence_barrier_init();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    while (u < u1 && u - u0 < 2) load_next();
  }
  if (warp == kMmaWarp) {
    tc5::alloc(smem_u32(tmem_slot), C::kTmemCols);
    tc5::relinquish_alloc_permit();
  }
  tc5::fence_before_thread_sync();
  __syncthreads();
  tc5::fence_after_thread_sync();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (std::is_void<T>::value && tid == 0 && blockIdx.x == 0 && a.amax) a.amax[0] = a.amax[1] = 0.0f;  // the second kernel joins its maxima to it
  const uint32_t tmem = *tmem_slot;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      while (u < u1) {
        if (u - u0 >= C::kStages && !tma::wait(empty0 + 8 * fill.slot, fill.phase ^ 1u)) {
          *stop = 1;
          break;
        }
        load_next();
      }
      // no copy may land after the block has gone: wait for the last fill of every stage
      const int64_t g = u - u0;
      for (int64_t j = g > C::kStages ? g - C::kStages : 0; j < g && kCopies; ++j)
        tma::wait(full0 + 8 * (int)(j % C::kStages), (uint32_t)(j / C::kStages) & 1u);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      Ring<C::kStages> r;
      Ring<2> acc;
      int64_t u = u0, tile = u0 / K.n;
      int kb = (int)(u0 - tile * K.n), n = 0;
      while (u < u1 && !*stop) {  // one tile's part
        const uint32_t shift = (uint32_t)(tile / cut.tiles_f * BN % 128 / 32);
        // its accumulator has been read out
        if (n >= 2 && !tma::wait(acce0 + 8 * acc.slot, acc.phase ^ 1u)) *stop = 1;
        bool fresh = true, last = false;
        for (; u < u1 && !last && !*stop; ++u, r.next()) {
          if (!tma::wait(sfr0 + 8 * r.slot, r.phase)) {
            *stop = 1;
            break;
          }
          tc5::fence_after_thread_sync();
          mma_stage<BN>(tmem + (uint32_t)(acc.slot * BN), tmem + 2 * BN + (uint32_t)r.slot * C::kSfCols, shift,
                        StageDesc(smem_u32(smem + r.slot * C::kStageBytes)), K.groups(kb), fresh);
          tc5::commit(empty0 + 8 * r.slot);
          fresh = false;
          last = ++kb == K.n;
        }
        if (*stop) break;
        kb = 0;
        ++tile;
        tc5::commit(accf0 + 8 * acc.slot);
        acc.next();
        ++n;
      }
      tc5::commit(drain);  // arrives when every MMA issued above has completed
    }
  } else if (warp >= kSfWarp0) {
    const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
    Ring<C::kStages> r;
    int kb = (int)(u0 % K.n);
    for (int64_t u = u0; u < u1; ++u, r.next()) {
      if (!__all_sync(0xFFFFFFFFu, tma::wait(full0 + 8 * r.slot, r.phase) && *stop == 0)) {
        if (lane == 0) *stop = 1;
        break;
      }
      put_scales<1>(tmem + quarter + 2 * BN + (uint32_t)r.slot * C::kSfCols, smem + r.slot * C::kStageBytes + C::kSfAt,
                    K.groups(kb), kb == K.n - 1 && K.tail, lane);
      tc5::fence_before_thread_sync();
      __syncwarp();
      if (lane == 0) arrive(sfr0 + 8 * r.slot);
      if (++kb == K.n) kb = 0;
    }
  } else {
    Ring<2> acc;
    const int64_t first = u0 / K.n;
    for (int64_t tile = first; tile * K.n < u1; ++tile, acc.next()) {
      const bool ready = tma::wait(accf0 + 8 * acc.slot, acc.phase);
      if (!__all_sync(0xFFFFFFFFu, ready && *stop == 0)) {
        if (lane == 0) *stop = 1;
        break;
      }
      tc5::fence_after_thread_sync();
      const int64_t t0 = tile / cut.tiles_f * BN;
      const int tokens = (int)(a.M - t0 < BN ? a.M - t0 : BN);
      float* out = nullptr;
      const int64_t n = tile % cut.tiles_f * kLaneRows + tid;
      float scale = 0.0f, bias = 0.0f;
      if constexpr (std::is_void<T>::value) {
        const int part = (int)blockIdx.x - cut.piece_of(tile * cut.steps);
        out = a.ws + ((tile * cut.most + part) * BN) * kLaneRows + tid;
      } else {
        scale = a.alpha_a[0] * a.alpha_b[0];
        if (a.bias && n < a.N) bias = load_as_f32(a.bias, n, a.bias_bf16);
      }
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        uint32_t v[16];
        ld_32x32b_x16(tmem + (uint32_t)(acc.slot * BN + c) + ((uint32_t)(32 * warp) << 16), v);
        tc5::wait_ld();
        if constexpr (std::is_void<T>::value) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < tokens) out[(int64_t)(c + i) * kLaneRows] = __uint_as_float(v[i]);
        } else if (n < a.N) {
          put_tokens<T>(a, t0 + c, n, tokens - c, reinterpret_cast<float*>(v), scale, bias);
        }
      }
      tc5::fence_before_thread_sync();
      __syncwarp();
      if (lane == 0) arrive(acce0 + 8 * acc.slot);
    }
  }
  __syncwarp();
  __syncthreads();
  const bool drained = tma::wait(drain, 0);
  if (tid == 0 && (*stop || !drained) && a.status) atomicExch(a.status, kStatusPipeline);
  tc5::fence_before_thread_sync();
  __syncthreads();
  if (warp == kMmaWarp) tc5::dealloc(tmem, C::kTmemCols);
}

// Epilogue of one output; returns the magnitude bits of the rounded d.
template <typename T>
__device__ __forceinline__ uint32_t put(const LinearArgs& a, int64_t m, int64_t n, float z) {
  if (a.z) static_cast<T*>(a.z)[m * a.ldz + n] = from_f32<T>(z);
  float d = act_value<T>(z, a.act);
  if (a.residual) d += to_f32(static_cast<const T*>(a.residual)[m * a.ldr + n]);
  const T o = from_f32<T>(d);
  static_cast<T*>(a.d)[m * a.ldd + n] = o;
  return abs_bits(to_f32(o));
}

// The pieces of output tile blockIdx.x added in order: a thread takes four features
// of a token, 32 apart, so that every access is a piece of one row whatever its
// alignment.
template <typename T>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearArgs a, const Cut cut, int bn) {
  const int64_t tile = blockIdx.x, f = tile % cut.tiles_f, tok = tile / cut.tiles_f;
  const int64_t m = tok * bn + (int64_t)blockIdx.y * blockDim.y + threadIdx.y, n = f * kLaneRows + threadIdx.x;
  const bool there = m < a.M && m < (tok + 1) * bn;
  float bias[4] = {};
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + 32 * i < a.N) bias[i] = load_as_f32(a.bias, n + 32 * i, a.bias_bf16);
  }
  const float scale = a.alpha_a[0] * a.alpha_b[0];
  const int parts = cut.piece_of((tile + 1) * cut.steps - 1) - cut.piece_of(tile * cut.steps) + 1;
  const float* in = a.ws + (tile * cut.most * bn + (m - tok * bn)) * kLaneRows + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t top = 0;
  if (there) {
    float v[4] = {};
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += in[(int64_t)p * bn * kLaneRows + 32 * i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + 32 * i < a.N) top = max(top, put<T>(a, m, n + 32 * i, fmaf(v[i], scale, bias[i])));
  }
  if (a.amax) {  // one warp per block: an atomic per warp cost 8 us for 1000 x 1000 outputs
    __shared__ uint32_t tops[8];
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (threadIdx.x == 0) tops[threadIdx.y] = top;
    __syncthreads();
    if (threadIdx.y == 0) put_amax(a.amax, threadIdx.x < blockDim.y ? tops[threadIdx.x] : 0u);
  }
}

Cut cut_of(int64_t M, int64_t N, int64_t K, int bn, bool whole) {
  Cut c;
  c.tiles_f = (N + kLaneRows - 1) / kLaneRows;
  c.tiles = c.tiles_f * ((M + bn - 1) / bn);
  c.steps = (int)((K + kBK - 1) / kBK);
  c.pieces = (int)std::min<int64_t>(152, whole ? c.tiles : c.tiles * c.steps);
  // a tile's steps meet at most this many pieces of at least floor(tiles * steps / pieces) steps
  const int64_t least = c.tiles * c.steps / c.pieces;
  c.most = whole ? 1 : (int)((c.steps + least - 2) / least + 1);
  c.whole = whole ? 1 : 0;
  return c;
}

template <int BN, typename T>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
  using C = Cfg<BN>;
  constexpr bool kWhole = !std::is_void<T>::value;
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
  const Cut cut = cut_of(a.M, a.N, a.K, BN, kWhole);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cut.pieces);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, wmap, xmap, cut);
  if (e != cudaSuccess || kWhole) return e;
  const int tokens = (int)std::min<int64_t>(a.M, BN);
  const int ty = tokens >= 8 ? 8 : tokens;
  cfg.gridDim = dim3((unsigned)cut.tiles, (unsigned)((tokens + ty - 1) / ty));
  cfg.blockDim = dim3(32, (unsigned)ty);
  cfg.dynamicSmemBytes = 0;
  return a.out_bf16 ? cudaLaunchKernelEx(&cfg, linear_join_kernel<bf16>, a, cut, BN)
                    : cudaLaunchKernelEx(&cfg, linear_join_kernel<float>, a, cut, BN);
}

template <int BN>
cudaError_t launch_cut(const LinearArgs& a, bool whole, cudaStream_t s) {
  if (!whole) return launch<BN, void>(a, s);
  return a.out_bf16 ? launch<BN, bf16>(a, s) : launch<BN, float>(a, s);
}

}  // namespace

int64_t split_workspace(int64_t M, int64_t N, int64_t K, int bn) {
  const Cut c = cut_of(M, N, K, bn, false);
  return c.tiles * c.most * bn * kLaneRows * 4;
}

cudaError_t launch_split(const LinearArgs& a, int bn, bool whole, cudaStream_t s) {
  switch (bn) {
    case 16: return launch_cut<16>(a, whole, s);
    case 32: return launch_cut<32>(a, whole, s);
    case 64: return launch_cut<64>(a, whole, s);
    default: return launch<128, void>(a, s);
  }
}

}  // namespace lin
}  // namespace nvfp4
