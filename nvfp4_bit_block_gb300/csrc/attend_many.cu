// attend_many.cu -- attention of sequences with many new rows (tokens times the query heads
// that share a key head) to the NVFP4 cache: prompts, or their parts.
//
// 4 D operations per row and visible key bound it: the tensor cores' rate.  A block takes 256
// rows of one key head as two tiles of 128 (one tile of 128 for D > 128, where TMEM holds no
// more) and walks over the visible keys, 64 at a time:
//   warps 8-11  bring codes and scales of a block of keys and values and leave them as fp16
//               in shared memory, in the layout that the tensor core reads (a code times its
//               scale is exact in fp16); done once for both tiles;
//   warp 12     issues S = Q K^T (shared memory to TMEM) and O += P V (P from TMEM);
//   warps 0-7   a thread for each row: S from TMEM, exponentials, P back to TMEM as fp16 in
//               the columns that S had.
// Each tile has two buffers of S: the next block's scores are formed while this one's rows are at
// their exponentials.  (128 keys at a time leave TMEM for one buffer and want registers moved to the
// rows: a row's next scores then wait for both products, and the three prompts of the largest measured
// case took as long.)
//
// Measured: prompts of 2731, 1818 and 905 tokens that end caches of 8192, 5454 and 2716 keys, 40 query
// heads on 8 of 128 values: 550 us, 1.08 PFLOP/s (56 % of the measured bf16 rate).  For each 64 keys a
// row takes about 1200 clocks, its block's products 1550 and the block 2360.  A product of 64 columns with
// both operands in shared memory takes the tensor core as long as one of 128, 64 clocks: 16 of S and 8 of O
// are 1536 where products of 128 columns throughout would be 1024.  The rest is the way from P's arrival to
// the issuing warp (270 clocks) and from the product's end back, twice for each block.  Keys of D 64 take
// 443 us (35 % of the rate), D 256 1421 (43 %: one tile, nothing to alternate with).
#include <cmath>

#include "attend.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace nvfp4 {
namespace attention {

namespace many {

constexpr int kRowWarps = 8, kFillWarps = 4;
constexpr int kMmaWarp = kRowWarps + kFillWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int BN = 64;  // keys of a block

template <int DP>
struct Shape {
  static constexpr int TILES = DP <= 128 ? 2 : 1;
  static constexpr int STAGES = DP <= 128 ? 4 : 2;  // blocks of keys, and of values
  static constexpr int Q_TILE = 128 * DP * 2;
  static constexpr int STAGE = BN * DP * 2;
  static constexpr int KS = 0;
  static constexpr int VS = STAGES * STAGE;
  static constexpr int QS = 2 * STAGES * STAGE;
  static constexpr int BARS = QS + TILES * Q_TILE;
  static constexpr int SMEM = BARS + 256 + 1024;  // 1024: what alignment may take
  static constexpr int UNITS = DP / 64;           // units of 32 values of a filling thread: every other one of a row
  static constexpr int O_COL = 256;               // TMEM: four buffers of S, then O
};

// mbarriers, eight bytes each
enum Bar { kKFull = 0, kKEmpty = 4, kVFull = 8, kVEmpty = 12, kSFull = 16, kPFull = 20, kPvDone = 24, kOFull = 26, kDrain = 28 };

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A warp's wait on a barrier: the same answer in every lane, false once the block has given up or
// after about a second.  What is there already costs a look and a vote: the warp that issues the
// products does little else, and with a clock read in each of its waits it was what bounded a block.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* stop) {
  const uint64_t t0 = tma::globaltimer();
  for (uint32_t i = 0; i < tma::kWaitLimitPolls; ++i) {
    const bool ok = tma::try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, ok)) return true;
    if ((i & 15u) == 15u && __any_sync(0xFFFFFFFFu, *stop != 0 || tma::globaltimer() - t0 > tma::kWaitLimitNs)) break;
  }
  *stop = 1;
  return false;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xFFFFFFFFu, tma::try_wait(bar, parity)) || wait_long(bar, parity, stop);
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// fp16 operands, fp32 sums: A (128 rows) and B with K contiguous, or B with its rows contiguous.
constexpr uint32_t idesc_f16(int N, bool b_rows) {
  return (1u << 4) | ((b_rows ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// A whole warp comes to these and its leader issues: without a branch around them the descriptors
// stay in uniform registers.  (Issued from inside `if (lane == 0)`, with descriptors formed for each
// product, one took 88 clocks where the tensor core takes 64.)  A descriptor's upper half is the same
// for all tiles of a kind; the lower one counts addresses in 16 bytes.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t upper, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n setp.ne.u32 q, %6, 0;\n"
      " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(upper), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t upper, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n setp.ne.u32 p, %5, 0;\n setp.ne.u32 q, %6, 0;\n"
      " mov.b64 y, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(upper), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elected() {  // 1 in one lane of the warp
  uint32_t r;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// One thread's part of a key or value row: units half, half + 2, .. of 32 values, as codes and scales.
template <int DP>
struct Raw {
  uint4 codes[Shape<DP>::UNITS];
  uint32_t scales[Shape<DP>::UNITS];  // two bytes of each
};

template <int DP>
__device__ __forceinline__ void load_raw(const uint8_t* codes, const uint8_t* scales, bool on, int half, int D, Raw<DP>& r) {
#pragma unroll
  for (int i = 0; i < Shape<DP>::UNITS; ++i) {
    const int u = half + 2 * i;
    const bool in = on && 32 * u < D;
    r.codes[i] = in ? *reinterpret_cast<const uint4*>(codes + 16 * u) : make_uint4(0, 0, 0, 0);
    r.scales[i] = in ? *reinterpret_cast<const uint16_t*>(scales + 2 * u) : 0;
  }
}

// .. and as fp16 in shared memory: row `row` of columns of 64 values, 16-byte pieces in the
// 128-byte swizzle.
template <int DP>
__device__ __forceinline__ void store_raw(uint8_t* stage, int row, int half, int D, const Raw<DP>& r) {
#pragma unroll
  for (int i = 0; i < Shape<DP>::UNITS; ++i) {
    const int u = half + 2 * i;
    if (32 * u >= D) continue;
    const uint32_t w[4] = {r.codes[i].x, r.codes[i].y, r.codes[i].z, r.codes[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t byte = r.scales[i] >> (8 * (k / 2)) & 0xFFu;
      const uint32_t f = scales2(byte * 0x101u);
      uint32_t h[4];
      codes8(w[k], h);
      const int piece = 4 * u + k;  // the two threads of a row write to different banks
      *reinterpret_cast<uint4*>(stage + piece / 8 * (BN * 128) + row * 128 + ((piece % 8) ^ (row & 7)) * 16) =
          make_uint4(h2_mul(h[0], f), h2_mul(h[1], f), h2_mul(h[2], f), h2_mul(h[3], f));
    }
  }
}

__device__ __forceinline__ int64_t tiles_of(const AttendArgs& a, int rows_per_block, int b, Sequence& s) {
  load_sequence(a.c, b, s);
  if (is_few(a, s)) return 0;
  return ((int64_t)s.rows * a.group + rows_per_block - 1) / rows_per_block;
}

template <int DP, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) many_kernel(AttendArgs a) {
  using S = Shape<DP>;
  constexpr int ROWS = 128 * S::TILES;
  extern __shared__ uint8_t dyn[];
  __shared__ Line line;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int stop;
  __shared__ int bad_page;
  const CacheView& c = a.c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  find_line<kThreads>(
      c, line, [&](int b) {
        Sequence s;
        return tiles_of(a, ROWS, b, s) * c.heads;
      },
      [&](int64_t) { return (int64_t)blockIdx.x; });
  if ((int64_t)blockIdx.x >= line.total) return;

  const int tid = threadIdx.x, warp = tid / 32, b = line.sequence, D = FULL ? DP : c.dim;
  uint8_t* sm = dyn + (1024 - smem_u32(dyn) % 1024) % 1024;
  const uint32_t base = smem_u32(sm), bars = base + S::BARS;
  auto bar = [&](int i) { return bars + 8 * i; };
  Sequence seq;
  const int64_t tiles = tiles_of(a, ROWS, b, seq);
  const int64_t unit = blockIdx.x - line.base;
  const int head = (int)(unit % c.heads);
  const int64_t row0 = (tiles - 1 - unit / c.heads) * ROWS;  // the tiles with the most keys first
  const int rows = (int)min((int64_t)ROWS, (int64_t)seq.rows * a.group - row0);
  const int nt = rows > 128 ? 2 : 1;
  const Keys<BN> keys = rows_keys<BN, uint64_t>(a, seq, (uint64_t)row0, rows);
  const int nb = keys.count;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      tma::mbar_init(bar(kKFull + i), 32 * kFillWarps);
      tma::mbar_init(bar(kVFull + i), 32 * kFillWarps);
      tma::mbar_init(bar(kKEmpty + i), 1);
      tma::mbar_init(bar(kVEmpty + i), 1);
      tma::mbar_init(bar(kSFull + i), 1);
      tma::mbar_init(bar(kPFull + i), 128);
    }
    for (int i = 0; i < 2; ++i) {
      tma::mbar_init(bar(kPvDone + i), 1);
      tma::mbar_init(bar(kOFull + i), 1);
    }
    tma::mbar_init(bar(kDrain), 1);
    tma::fence_barrier_init();
    stop = 0;
    bad_page = 0;
  }
  if (warp == kMmaWarp) {
    tc5::alloc(smem_u32(&tmem_slot), 512);
    tc5::relinquish_alloc_permit();
  }

  // queries: a thread for each row
  const int tile = warp / 4, row_in = tile * 128 + tid % 128;
  const bool is_row = warp < 4 * nt, on = is_row && row_in < rows;
  const int64_t row = row0 + row_in;
  const int64_t token = on ? seq.first + row / a.group : 0;
  const int qh = on ? head * a.group + (int)(row % a.group) : 0;
  const int p = seq.length - seq.rows + (int)(row / a.group);  // position
  float f = 0.0f;
  if (is_row) {
    const bf16* q = static_cast<const bf16*>(a.q.p) + token * a.q.ts + (int64_t)qh * a.q.hs;
    const bool vec = rows_at_16(a.q);
    uint32_t top = 0;
    if (on) {
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 w = load_query8(q + 8 * i, vec);
        top = larger_magnitude(larger_magnitude(larger_magnitude(larger_magnitude(top, w.x), w.y), w.z), w.w);
      }
    }
    // scores to base 2 are f * S with f > 0: the scale's sign goes into the queries, and where it
    // vanishes f is the smallest number, so that -Inf stays -Inf
    f = a.scale * c.alpha[0] * layer::kLog2e * query_up(top);
    const float down = f < 0.0f ? -query_down(top) : query_down(top);
    f = fmaxf(fabsf(f), 0x1p-126f);
    uint8_t* qs = sm + S::QS + tile * S::Q_TILE;
    const int r = tid % 128;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const uint4 w = on ? load_query8(q + 8 * i, vec) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(qs + i / 8 * (128 * 128) + r * 128 + ((i % 8) ^ (r & 7)) * 16) =
          make_uint4(pack_h2(bf16_lo(w.x) * down, bf16_hi(w.x) * down), pack_h2(bf16_lo(w.y) * down, bf16_hi(w.y) * down),
                     pack_h2(bf16_lo(w.z) * down, bf16_hi(w.z) * down), pack_h2(bf16_lo(w.w) * down, bf16_hi(w.w) * down));
    }
    fence_async_smem();
  }
  tc5::fence_before_thread_sync();
  __syncthreads();
  tc5::fence_after_thread_sync();
  // Only now may the next kernel begin: one that takes TMEM in its setup, before it waits for this one,
  // would otherwise hold on an SM what this block still has to get there, and each would wait for the other.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // pages out of range, all of them before any key is used: their keys are hidden
  {
    bool bad = false;
    for (int i = tid; i < nb; i += kThreads) {
      const int64_t key = (int64_t)keys.chunk(i) * BN, end = min(key + BN, (int64_t)seq.length);
      for (int64_t j = key; j < end; j = (j / c.page_size + 1) * c.page_size) bad |= page_of(c, b, (int)j) < 0;
    }
    if (bad) {
      bad_page = 1;
      set_status(c.status, NVFP4_ERR_INDEX);
    }
  }
  __syncthreads();
  const uint32_t tmem = tmem_slot;
  const bool holes = bad_page != 0;

  if (warp < kRowWarps) {
    if (is_row) {
      const uint32_t at = tmem + ((uint32_t)(warp % 4 * 32) << 16), o_at = at + S::O_COL + tile * D;
      float m = -INFINITY;
      float2 l0 = make_float2(0.0f, 0.0f), l1 = l0;
      const int hi = a.causal ? min(p, seq.length - 1) : seq.length - 1;  // the last key that this row sees
      const int64_t lo = a.causal && a.window ? (int64_t)p - a.window : -1;  // keys up to this one lie before the window
      bool got = nb > 0;
      for (int i = 0; i < nb; ++i) {
        const int buf = 2 * tile + (i & 1);
        if (!(got = warp_wait(bar(kSFull + buf), (i >> 1) & 1, &stop))) break;
        tc5::fence_after_thread_sync();
        const uint32_t s_at = at + BN * buf;
        const int key = keys.chunk(i) * BN;
        const bool part = !keys.all_visible(key);
        // columns up to last, of them those behind before and those below first
        const int last = hi - key, before = (int)max(lo - key, (int64_t)-1), first = a.sinks - key;
        if (holes) {  // pages hold 16 keys at least, and are out of range for every row
          for (int x = 0; x < BN; x += 16) {
            if (key + x >= seq.length || page_of(c, b, key + x) >= 0) continue;
            uint32_t none[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) none[y] = 0xFF800000u;
            st_x16(s_at + x, none);
          }
          tc5::wait_st();
        }
        float s[BN];
#pragma unroll
        for (int x = 0; x < BN; x += 32) tc5::ld_32x32b_x32(s_at + x, reinterpret_cast<uint32_t*>(s + x));
        tc5::wait_ld();
        if (part) {
#pragma unroll
          for (int x = 0; x < BN; ++x) s[x] = (x <= last) & ((x > before) | (x < first)) ? s[x] : -INFINITY;
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int x = 4; x < BN; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) top[y] = x + y + 4 < BN ? fmaxf(top[y], fmaxf(s[x + y], s[x + y + 4])) : fmaxf(top[y], s[x + y]);
        float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f, g = f;
        // A score times f and what is taken off it are one rounding, the maximum has one of its own: where
        // a step of that is no longer small, the row's scores are rounded alike, so that no weight passes
        // 2^15.  (Always so, the largest measured case takes 570 us and not 548.)
        const bool coarse = fabsf(high) > 0x1p20f && fabsf(high) < INFINITY;
        if (__any_sync(0xFFFFFFFFu, coarse)) {
          g = coarse ? 1.0f : f;
          const float once = coarse ? f : 1.0f;
#pragma unroll
          for (int x = 0; x < BN; ++x) s[x] *= once;
        }
        const bool up = high - m > kMoves;
        if (__any_sync(0xFFFFFFFFu, up)) {
          const float d = up ? layer::ex2(m - (high - kLift)) : 1.0f;
          if (up) m = high - kLift;
          l0 = mul2(l0, make_float2(d, d));
          l1 = mul2(l1, make_float2(d, d));
          if (i > 0) {  // what O holds of the blocks before, once the last of them is in
            // (parity tells that phase from its neighbours alone: S came after the product before it)
            if (!(got = warp_wait(bar(kPvDone + tile), (i - 1) & 1, &stop))) break;
            tc5::fence_after_thread_sync();
#pragma unroll 1
            for (int x = 0; x < D; x += 16) {
              uint32_t o[16];
              ld_x16(o_at + x, o);
              tc5::wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * d);
              st_x16(o_at + x, o);
            }
          }
        }
        const float z = m == -INFINITY ? 0.0f : -m;
        const float2 f2 = make_float2(g, g), z2 = make_float2(z, z);
#pragma unroll
        for (int x = 0; x < BN; x += 32) {
          uint32_t h[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float2 t = fma2(make_float2(s[x + 2 * y], s[x + 2 * y + 1]), f2, z2);
            const float2 e = make_float2(layer::ex2(t.x), layer::ex2(t.y));
            if (y & 1)
              l1 = add2(l1, e);
            else
              l0 = add2(l0, e);
            h[y] = pack_h2(e.x, e.y);
          }
          st_x16(s_at + x / 2, h);
        }
        tc5::wait_st();
        tc5::fence_before_thread_sync();
        arrive(bar(kPFull + buf));
      }
      // the result
      const float l = (l0.x + l0.y) + (l1.x + l1.y);
      const float share = l != 0.0f ? c.alpha[1] / l : 0.0f;
      if (on && a.lse) a.lse[token * a.Hq + qh] = row_lse(m, l);
      got = got && warp_wait(bar(kOFull + tile), 0, &stop);
      tc5::fence_after_thread_sync();
      bf16* out = static_cast<bf16*>(a.o.p) + token * a.o.ts + (int64_t)qh * a.o.hs;
      const bool vec = rows_at_16(a.o);
      for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        __syncwarp();  // lanes without a row have not stored
        if (got) {
          tc5::ld_32x32b_x32(o_at + x, o);
          tc5::wait_ld();
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0;
        }
        if (!on) continue;
        uint32_t h[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const __nv_bfloat162 v =
              __floats2bfloat162_rn(__uint_as_float(o[2 * y]) * share, __uint_as_float(o[2 * y + 1]) * share);
          h[y] = *reinterpret_cast<const uint32_t*>(&v);
        }
        if (vec) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
            reinterpret_cast<uint4*>(out + x)[y] = make_uint4(h[4 * y], h[4 * y + 1], h[4 * y + 2], h[4 * y + 3]);
        } else {
          uint16_t* e = reinterpret_cast<uint16_t*>(out + x);
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            e[2 * y] = (uint16_t)h[y];
            e[2 * y + 1] = (uint16_t)(h[y] >> 16);
          }
        }
      }
    }
  } else if (warp < kMmaWarp) {
    const int t = tid - 32 * kRowWarps, r = t / 2, half = t % 2;
    const int64_t hc = (int64_t)head * c.ch, hs = (int64_t)head * c.sh;
    // Keys of the next block are on their way while this block's values are unpacked, then its values;
    // its page is looked up a block before.
    Raw<DP> k, v;
    int64_t co = 0, so = 0;  // where this thread's row lies
    int page = -1;
    uint32_t in = 0;
    auto look = [&](int i) {
      const int64_t key = (int64_t)keys.chunk(i) * BN + r;
      page = key < seq.length ? c.table[(int64_t)b * c.table_stride + (uint32_t)key / (uint32_t)c.page_size] : -1;
      in = (uint32_t)key % (uint32_t)c.page_size;
    };
    auto place = [&]() {
      const bool on = (uint32_t)page < (uint32_t)c.pages;
      co = hc + (int64_t)((uint64_t)(on ? page : 0) * c.cp + (uint64_t)in * c.cr);
      so = hs + (int64_t)((uint64_t)(on ? page : 0) * c.sp + (uint64_t)in * c.sr);
      return on;
    };
    bool on = false;
    if (nb > 0) {
      look(0);
      on = place();
      load_raw<DP>(c.kc + co, c.ks + so, on, half, D, k);
      load_raw<DP>(c.vc + co, c.vs + so, on, half, D, v);
      if (nb > 1) look(1);
    }
    for (int i = 0; i < nb; ++i) {
      const int st = i % S::STAGES, round = i / S::STAGES;
      if (round > 0 && !warp_wait(bar(kKEmpty + st), (round - 1) & 1, &stop)) break;
      store_raw<DP>(sm + S::KS + st * S::STAGE, r, half, D, k);
      fence_async_smem();
#ifdef NVFP4_TEST_NO_COPIES  // the test build's keys come no more from the fifth block on
      if (i < 4)
#endif
        arrive(bar(kKFull + st));
      if (i + 1 < nb) {
        on = place();
        load_raw<DP>(c.kc + co, c.ks + so, on, half, D, k);
      }
      if (round > 0 && !warp_wait(bar(kVEmpty + st), (round - 1) & 1, &stop)) break;
      store_raw<DP>(sm + S::VS + st * S::STAGE, r, half, D, v);
      fence_async_smem();
      arrive(bar(kVFull + st));
      if (i + 1 < nb) {
        load_raw<DP>(c.vc + co, c.vs + so, on, half, D, v);
        if (i + 2 < nb) look(i + 2);
      }
    }
  } else {
    if (nb > 0) {
      const uint32_t leader = elected();
      constexpr uint32_t qk = idesc_f16(BN, false);
      const uint32_t pv = FULL ? idesc_f16(DP, true) : idesc_f16(D, true);
      const int steps = FULL ? DP / 16 : D / 16;
      // descriptors count addresses in 16 bytes: what a tile, a stage and a step of K add to them
      const uint64_t q0 = tc5::smem_desc(base + S::QS, 16, 1024, tc5::kLayoutSwizzle128B);
      const uint64_t k0 = tc5::smem_desc(base + S::KS, 16, 1024, tc5::kLayoutSwizzle128B);
      const uint64_t v0 = tc5::smem_desc(base + S::VS, BN * 128, 1024, tc5::kLayoutSwizzle128B);
      // Four blocks in a row are written out, so that stages, buffers and most parities are constants:
      // u is a block's number modulo 4, fours that of the fours before it modulo 2.
      auto product_qk = [&](int t, int u, uint32_t fours) {
        const int st = u % S::STAGES, buf = 2 * t + (u & 1);
        if (t == 0 && !warp_wait(bar(kKFull + st), S::STAGES == 4 ? fours : u >> 1, &stop)) return false;
        tc5::fence_after_thread_sync();
#pragma unroll
        for (int x = 0; x < DP / 16; ++x)
          if (FULL || x < steps)
            mma_ss(leader, tmem + BN * buf, (uint32_t)q0 + (t * S::Q_TILE + x / 4 * (128 * 128) + x % 4 * 32) / 16,
                   (uint32_t)k0 + (st * S::STAGE + x / 4 * (BN * 128) + x % 4 * 32) / 16, (uint32_t)(q0 >> 32), qk, x > 0);
        commit(leader, bar(kSFull + buf));
        if (t == nt - 1) commit(leader, bar(kKEmpty + st));
        return true;
      };
      auto product_pv = [&](int t, int u, uint32_t fours, bool first, bool last) {
        const int st = u % S::STAGES, buf = 2 * t + (u & 1);
        if (t == 0 && !warp_wait(bar(kVFull + st), S::STAGES == 4 ? fours : u >> 1, &stop)) return false;
        if (!warp_wait(bar(kPFull + buf), u >> 1, &stop)) return false;
        tc5::fence_after_thread_sync();
#pragma unroll
        for (int x = 0; x < BN / 16; ++x)
          mma_ts(leader, tmem + S::O_COL + t * D, tmem + BN * buf + 8 * x, (uint32_t)v0 + (st * S::STAGE + x * 2048) / 16,
                 (uint32_t)(v0 >> 32), pv, !first || x > 0);
        commit(leader, bar(kPvDone + t));
        if (last) commit(leader, bar(kOFull + t));
        if (t == nt - 1) commit(leader, bar(kVEmpty + st));
        return true;
      };
      // a buffer of S is free for the block after next once its P has been used: products run in order
      bool ok = true;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && u < nb && t < nt) ok = product_qk(t, u, 0);
      uint32_t fours = 0;
      for (int i = 0; ok && i < nb; i += 4, fours ^= 1) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (ok && i + u < nb && t < nt) {
              ok = product_pv(t, u, fours, i + u == 0, i + u == nb - 1);
              if (ok && i + u + 2 < nb) ok = product_qk(t, (u + 2) % 4, u < 2 ? fours : fours ^ 1);
            }
      }
      // What has been issued is waited for also where the block has given up: the tensor memory that it
      // writes is freed behind this.
      commit(leader, bar(kDrain));
      if (!tma::wait(bar(kDrain), 0)) stop = 1;
    }
  }
  __syncwarp();
  tc5::fence_before_thread_sync();
  __syncthreads();
  tc5::fence_after_thread_sync();
  if (warp == kMmaWarp) tc5::dealloc(tmem, 512);
  if (tid == 0 && stop) set_status(c.status, NVFP4_ERR_PIPELINE);
}

template <int DP, bool FULL>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  using S = Shape<DP>;
  const cudaError_t e = cudaFuncSetAttribute(many_kernel<DP, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  // as many blocks as the batch can have tiles: one more for each sequence that is not surely few
  const int64_t rows = (int64_t)a.c.T * a.group, sequences = rows / (surely_few(a) + 1);
  const int64_t tiles = rows / (128 * S::TILES) + (sequences < a.c.sequences ? sequences : a.c.sequences);
  const int64_t blocks = tiles * a.c.heads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_early(many_kernel<DP, FULL>, dim3((unsigned)blocks), kThreads, S::SMEM, s, a);
}

}  // namespace many
}  // namespace attention

cudaError_t launch_attend_many(const AttendArgs& a, cudaStream_t s) {
  using namespace attention;
  if (a.c.dim <= 64) return a.c.dim == 64 ? many::launch<64, true>(a, s) : many::launch<64, false>(a, s);
  if (a.c.dim <= 128) return a.c.dim == 128 ? many::launch<128, true>(a, s) : many::launch<128, false>(a, s);
  return a.c.dim == 256 ? many::launch<256, true>(a, s) : many::launch<256, false>(a, s);
}

}  // namespace nvfp4
