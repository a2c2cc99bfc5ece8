// attend_few.cu -- attention of sequences with few new rows (tokens times the query heads
// that share a key head) to the NVFP4 cache: the next token, or a few drafted ones.
//
// The cache's bytes are the floor: 9/16 byte per value, read once for all heads of a group.
// A unit of work is a tile of 8 or 16 rows of one key head; its visible keys are cut into
// steps of 64 and the steps of all units form one line that is cut into equal pieces, one per
// block, so that one long sequence and many short ones fill the GPU alike.  Pieces that are part
// of a unit leave (m, l, o) in the workspace and a second kernel joins them in order.
//
// Within a step each of a block's four warps takes 16 keys, whose bytes come by asynchronous
// copies into the warp's own ring in shared memory, a few chunks ahead (with the next chunk on
// its way in registers instead, each SM had 20 KB in flight where the latency wants 45).  From
// there to the output they stay in registers, as the first operand of m16n8k16 products in fp16
// with fp32 sums: S^T = K Q^T for 16 keys and 8 rows, O^T += V^T P^T for 16 values and 8 rows.  (With
// the rows first, a tile has 16 of them and most are empty: twice the products and registers for o.)
// A code times its scale has at most 6 significant bits within 2^-10..2688, so it is exact in
// fp16; queries are scaled by a power of two per row.  Which of a product's k's (and of its 16
// values) a value counts as is free, as long as both operands agree: each lane loads bytes that
// lie side by side and uses them where they are.  Lane (g, q) = (lane / 4, lane % 4) has for key
// rows g and 8 + g the q-th quarter of the values, and for the value rows 2q, 2q + 1, 8 + 2q,
// 9 + 2q the g-th eighth.  P leaves its product with keys along g and rows along q and enters the
// next one the other way round: movmatrix turns it.
//
// Measured: the next token of 48 sequences of up to 16384 keys, 40 query heads on 8 of 128 values: 132 us
// for 509 MB, 3.9 TB/s (57 % of the copy rate).  About 430 instructions for 16 keys, 60 % of the issue
// slots busy with 16 warps on an SM.  Half of them unpack: 72 conversions and 64 products by scales, two
// clocks each.  One token of 700 keys: 12 us with its host side.
#include <cmath>

#include "attend.cuh"

namespace nvfp4 {
namespace attention {

constexpr int kWarps = 4;
constexpr int kThreadsFew = 32 * kWarps;

template <int DP, int NT>
struct Few {
  static constexpr int ROWS = 8 * NT;   // of a tile
  static constexpr int KW = DP / 32;    // words of a lane's part of a key (DP / 4 values)
  static constexpr int KS = DP / 64;    // its scales
  static constexpr int VN = DP / 8;     // values of a lane's part of a value row
  static constexpr int VW = VN / 8;     // words of it
  // A chunk in a warp's ring: rows of codes (16 bytes apart in their banks), then scales as the
  // cache has them; of keys, then of values.
  static constexpr int CODE_ROW = DP / 2 + 16;
  static constexpr int CODES = 16 * CODE_ROW, SCALES = 16 * (DP / 16);
  static constexpr int STAGE = 2 * (CODES + SCALES);
  static constexpr int STAGES = DP == 256 ? 3 : 4;
  static constexpr int COPIES = DP / 64;  // 16-byte pieces of a lane in 16 rows of codes
  // Queries stay in registers where they are few.
  static constexpr bool Q_SHARED = DP * NT > 128;
  // shared memory: the rings, and in the end o of the four warps in their place; m and l; queries
  static constexpr int O_ROW = DP + 2;
  static constexpr int RING = kWarps * STAGES * STAGE, O = kWarps * ROWS * O_ROW * 4;
  static constexpr int ML = RING > O ? RING : O;
  static constexpr int QS = ML + 2 * kWarps * ROWS * 4;
  static constexpr int SMEM = QS + (Q_SHARED ? DP / 32 * NT * 32 * 16 : 0);
  // Blocks: as many as an SM holds of them by registers, on every SM.
  static constexpr int PER_SM = DP == 64 ? (NT == 1 ? 5 : 4) : DP == 128 ? (NT == 1 ? 4 : 3) : NT == 1 ? 3 : 2;
  static constexpr int BLOCKS = 152 * PER_SM;
  // The workspace: a FewHead for each block, then two slots (o, m and l of a tile) for each.
  static constexpr int64_t SLOT = ROWS * DP + 2 * ROWS;
  static constexpr int64_t HEADS = (BLOCKS * (int64_t)sizeof(FewHead) / 4 + 3) / 4 * 4;
  static constexpr int64_t FLOATS = HEADS + 2 * BLOCKS * SLOT;
};

// One lane's bytes of 16 keys, and of 16 values; scale bytes, first lowest.
template <int DP>
struct RawKeys {
  uint32_t w[2][DP / 32], s[2];
};
template <int DP>
struct RawValues {
  uint32_t w[4][DP / 64], s[4];
};

__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of fp16, two of row lane / 4 in each lane, to its transpose.
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// What lane (g, q) needs of a chunk in the ring; FULL: D is DP, else parts beyond D are zeros.
template <int DP, bool FULL>
__device__ __forceinline__ void take_keys(const uint8_t* stage, int D, int g, int q, RawKeys<DP>& r) {
  using F = Few<DP, 1>;
  const int row = FULL ? DP / 16 : D / 16;
  const uint8_t* p = stage + g * F::CODE_ROW + q * (DP / 8);
  const uint8_t* s = stage + 2 * F::CODES + g * row + q * F::KS;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    r.s[t] = 0;
    if constexpr (DP == 64) {
      if (FULL || q * 16 < D) {
        const uint2 w = *reinterpret_cast<const uint2*>(p + 8 * t * F::CODE_ROW);
        r.w[t][0] = w.x;
        r.w[t][1] = w.y;
        r.s[t] = s[8 * t * row];
      } else {
        r.w[t][0] = r.w[t][1] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < F::KW / 4; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (FULL || q * (DP / 4) + 32 * i < D) {
          w = *reinterpret_cast<const uint4*>(p + 8 * t * F::CODE_ROW + 16 * i);
          r.s[t] |= (uint32_t)*reinterpret_cast<const uint16_t*>(s + 8 * t * row + 2 * i) << (16 * i);
        }
        r.w[t][4 * i] = w.x;
        r.w[t][4 * i + 1] = w.y;
        r.w[t][4 * i + 2] = w.z;
        r.w[t][4 * i + 3] = w.w;
      }
    }
  }
}
template <int DP, bool FULL>
__device__ __forceinline__ void take_values(const uint8_t* stage, int D, int g, int q, RawValues<DP>& r) {
  using F = Few<DP, 1>;
  const int row = FULL ? DP / 16 : D / 16;
  const uint8_t* p = stage + F::CODES + 2 * q * F::CODE_ROW + g * (DP / 16);
  const uint8_t* s = stage + 2 * F::CODES + F::SCALES + 2 * q * row + g * F::VN / 16;
  const bool on = FULL || g * F::VN < D;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int at = 8 * (t / 2) + t % 2;
    r.s[t] = 0;
#pragma unroll
    for (int i = 0; i < F::VW; ++i) r.w[t][i] = 0;
    if (!on) continue;
    const uint8_t* w = p + at * F::CODE_ROW;
    if constexpr (DP == 64) {
      r.w[t][0] = *reinterpret_cast<const uint32_t*>(w);
      r.s[t] = s[at * row];
    } else if constexpr (DP == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(w);
      r.w[t][0] = v.x;
      r.w[t][1] = v.y;
      r.s[t] = s[at * row];
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(w);
      r.w[t][0] = v.x;
      r.w[t][1] = v.y;
      r.w[t][2] = v.z;
      r.w[t][3] = v.w;
      r.s[t] = *reinterpret_cast<const uint16_t*>(s + at * row);
    }
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's share of the copies of one chunk: what it adds to where the chunk begins.
template <int DP, bool FULL>
struct Copies {
  using F = Few<DP, 1>;
  const uint8_t* codes[F::COPIES];  // keys'
  int64_t to_values;                // .. and values' from there
  const uint8_t* scales;            // keys' in lanes 0-15, values' in the others
  uint32_t code_at[F::COPIES], scale_at;  // in a stage of the ring; ~0: none
  __device__ __forceinline__ Copies(const CacheView& c, int lane, int h, bool dense) {
    const int pieces = FULL ? DP / 32 : c.dim / 32;  // of a row
#pragma unroll
    for (int i = 0; i < F::COPIES; ++i) {
      const int x = lane + 32 * i, row = x / pieces, piece = x % pieces;
      codes[i] = c.kc + h * c.ch + (uint64_t)row * c.cr + 16 * piece;
      code_at[i] = row < 16 ? row * F::CODE_ROW + 16 * piece : ~0u;
    }
    to_values = c.vc - c.kc;
    const int half = lane / 16, x = lane % 16, bytes = FULL ? DP / 16 : c.dim / 16;
    scales = (half ? c.vs : c.ks) + h * c.sh + (dense ? (uint64_t)(16 * x) : (uint64_t)x * c.sr);
    scale_at = 2 * F::CODES + half * F::SCALES + (dense ? 16 * x : x * bytes);
    if (dense && x >= bytes) scale_at = ~0u;
  }
  // code, scale: the chunk's offsets; dense: its 16 rows of scales lie side by side, at 16 bytes
  __device__ __forceinline__ void issue(const CacheView& c, uint64_t code, uint64_t scale, uint32_t stage, bool dense) const {
#pragma unroll
    for (int i = 0; i < F::COPIES; ++i) {
      if (!FULL && code_at[i] == ~0u) continue;
      const uint8_t* p = codes[i] + code;
      copy16(stage + code_at[i], p);
      copy16(stage + F::CODES + code_at[i], p + to_values);
    }
    if (dense) {
      if ((FULL && DP == 256) || scale_at != ~0u) copy16(stage + scale_at, scales + scale);
    } else {
      const uint8_t* p = scales + scale;
      for (int i = 0; i < (FULL ? DP / 16 : c.dim / 16); i += 2)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + scale_at + i), "h"(*reinterpret_cast<const uint16_t*>(p + i)) : "memory");
    }
  }
};

// A warp's way along its chunks, four apart: which page holds the chunk, and where in it.
struct Walk {
  int chunk, slot, in;  // in: chunks of the page before it
  __device__ __forceinline__ void begin(int c, int per_page) {
    chunk = c;
    slot = c / per_page;
    in = c - slot * per_page;
  }
  __device__ __forceinline__ void go(int c, int per_page) {
    if (c != chunk + kWarps) {  // from the first keys to the window
      begin(c, per_page);
      return;
    }
    chunk = c;
    in += kWarps;
    while (in >= per_page) {
      in -= per_page;
      ++slot;
    }
  }
};

// A lane's part of a row's queries in fp16, their sign turned if `minus`; returns what undoes their
// scaling.
template <int DP>
__device__ __forceinline__ float load_query(const AttendArgs& a, bool vec, bool on, int64_t token, int head, bool minus,
                                            uint32_t* h) {
  constexpr int N = DP / 4;  // this lane's values
  const int q = threadIdx.x % 4, D = a.c.dim;
  const bf16* p = static_cast<const bf16*>(a.q.p) + token * a.q.ts + (int64_t)head * a.q.hs + q * N;
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint4 w = on && q * N + 8 * i < D ? load_query8(p + 8 * i, vec) : make_uint4(0, 0, 0, 0);
    h[4 * i] = w.x;
    h[4 * i + 1] = w.y;
    h[4 * i + 2] = w.z;
    h[4 * i + 3] = w.w;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) top = larger_magnitude(top, h[i]);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float down = minus ? -query_down(top) : query_down(top);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) h[i] = pack_h2(bf16_lo(h[i]) * down, bf16_hi(h[i]) * down);
  return query_up(top);
}

// The keys of a tile of a sequence's rows, in chunks of 16, and the steps of 64 that all its
// tiles make for one key head.
template <int ROWS>
__device__ __forceinline__ Keys<16> tile_keys(const AttendArgs& a, const Sequence& s, int tile) {
  return rows_keys<16, uint32_t>(a, s, ROWS * tile, min(ROWS, s.rows * a.group - ROWS * tile));
}
template <int ROWS>
__device__ __forceinline__ int64_t sequence_steps(const AttendArgs& a, const Sequence& s) {
  int64_t n = 0;
  for (int r = 0; ROWS * r < s.rows * a.group; ++r) n += tile_keys<ROWS>(a, s, r).steps();
  return n;
}
__device__ __forceinline__ void load_few(const AttendArgs& a, int b, Sequence& s) {
  load_sequence(a.c, b, s);
  if (!is_few(a, s)) s.rows = 0;
}

template <int DP, int NT, bool FULL>
__global__ void __launch_bounds__(kThreadsFew, Few<DP, NT>::PER_SM) few_kernel(AttendArgs a) {
  using F = Few<DP, NT>;
  constexpr int ROWS = F::ROWS;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Line line;
  const CacheView& c = a.c;
  after_previous();
  const float alpha_v = c.alpha[1], scale = a.scale * c.alpha[0] * layer::kLog2e;  // on their way with the lengths
  if (blockIdx.x == 0) check_batch(c);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, q = lane % 4;
  float* os = reinterpret_cast<float*>(sm);          // [warps][ROWS][O_ROW]
  float* ms = reinterpret_cast<float*>(sm + F::ML);  // [warps][ROWS]
  float* ls = ms + kWarps * ROWS;                    // [warps][ROWS]
  uint4* qs = reinterpret_cast<uint4*>(sm + F::QS);  // [KW][NT][32], Q_SHARED
  uint8_t* ring = sm + warp * F::STAGES * F::STAGE;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  find_line<kThreadsFew>(
      c, line, [&](int b) {
        Sequence s;
        load_few(a, b, s);
        return sequence_steps<ROWS>(a, s) * c.heads;
      },
      [&](int64_t total) { return Pieces(total, gridDim.x).begin(blockIdx.x); });
  const Pieces pieces(line.total, gridDim.x);
  int64_t w = pieces.begin(blockIdx.x);
  const int64_t w_end = pieces.begin(blockIdx.x + 1);
  FewHead* heads = reinterpret_cast<FewHead*>(a.ws);
  if (threadIdx.x == 0) heads[blockIdx.x].last = -1;
  if (w >= w_end) return;

  Sequence seq;
  int b = line.sequence;
  load_few(a, b, seq);
  int64_t base = line.base;  // where sequence b begins on the line
  const bool vec = rows_at_16(a.q);
  const bool o_pairs = reinterpret_cast<uintptr_t>(a.o.p) % 4 == 0 && a.o.ts % 2 == 0 && a.o.hs % 2 == 0;
  const bool dense = c.sr == c.dim / 16 &&
                     (reinterpret_cast<uintptr_t>(c.ks) | reinterpret_cast<uintptr_t>(c.vs) | c.sp | c.sh) % 16 == 0;

  while (w < w_end) {
    // the unit that w is in
    int64_t per_head = sequence_steps<ROWS>(a, seq);
    while (w >= base + per_head * c.heads) {
      base += per_head * c.heads;
      load_few(a, ++b, seq);
      per_head = sequence_steps<ROWS>(a, seq);
    }
    const int64_t in = w - base;  // of the sequence
    const int h = (in | per_head) <= UINT32_MAX ? (int)((uint32_t)in / (uint32_t)per_head) : (int)(in / per_head);
    int64_t u0 = base + h * per_head;
    int r = 0;
    Keys<16> keys = tile_keys<ROWS>(a, seq, 0);
    while (w >= u0 + keys.steps()) {
      u0 += keys.steps();
      keys = tile_keys<ROWS>(a, seq, ++r);
    }
    const int64_t u1 = u0 + keys.steps();
    const int s_begin = (int)(w - u0), s_end = (int)((w_end < u1 ? w_end : u1) - u0);
    const int rows = min(ROWS, seq.rows * a.group - ROWS * r);

    __syncthreads();  // the part before is read
    // This warp's chunks are those of i, i + 4, ..; the copies are STAGES - 1 of them ahead, the
    // page of the next to be copied one more.
    const int per_page = c.page_size / 16, i_end = min(keys.count, 4 * s_end);
    const int32_t* table = c.table + (int64_t)b * c.table_stride;
    const Copies<DP, FULL> copies(c, lane, h, dense);
    Walk at;
    int ahead = 4 * s_begin + warp, page = -1, put = 0;
    uint32_t there = 0;  // by stage: whether the chunk's page is in range
    if (ahead < i_end) {
      at.begin(keys.chunk(ahead), per_page);
      page = __ldg(table + at.slot);
    }
    auto copy = [&]() {
      if (ahead < i_end) {
        there &= ~(1u << put);
        if ((uint32_t)page < (uint32_t)c.pages) {
          const uint32_t pg = page, row = 16 * at.in;
          const uint64_t codes = (uint64_t)pg * c.cp + (uint64_t)row * c.cr, scales = (uint64_t)pg * c.sp + (uint64_t)row * c.sr;
          copies.issue(c, codes, scales, ring_at + put * F::STAGE, dense);
          there |= 1u << put;
        } else {
          set_status(c.status, NVFP4_ERR_INDEX);
        }
        put = (put + 1) % F::STAGES;
        ahead += kWarps;
        if (ahead < i_end) {
          at.go(keys.chunk(ahead), per_page);
          page = __ldg(table + at.slot);
        }
      }
      copies_end();
    };
#pragma unroll
    for (int x = 0; x < F::STAGES - 1; ++x) copy();
    // queries: rows g of each eight; scores and o: rows 2q and 2q + 1
    uint32_t qf[NT][F::KW * 4];
    float f[NT][2];
    int p[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = ROWS * r + 8 * n + g;
      const bool on = 8 * n + g < rows;
      const float up = load_query<DP>(a, vec, on, (int64_t)seq.first + (on ? row / a.group : 0),
                                      h * a.group + (on ? row % a.group : 0), scale < 0.0f, qf[n]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // scores to base 2 are f * S with f > 0: the scale's sign is in the queries, and where it vanishes
        // f is the smallest number, so that -Inf stays -Inf
        f[n][e] = fmaxf(fabsf(scale) * __shfl_sync(0xFFFFFFFFu, up, 8 * q + 4 * e), 0x1p-126f);
        const int x = 8 * n + 2 * q + e;
        p[n][e] = seq.length - seq.rows + (x < rows ? (ROWS * r + x) / a.group : 0);
      }
    }
    if constexpr (F::Q_SHARED) {
      if (warp == 0)
#pragma unroll
        for (int x = 0; x < F::KW; ++x)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            qs[(x * NT + n) * 32 + lane] = make_uint4(qf[n][4 * x], qf[n][4 * x + 1], qf[n][4 * x + 2], qf[n][4 * x + 3]);
      __syncthreads();
    }

    float o[F::VN / 2][NT][4] = {};
    float m[NT][2], z[NT][2], l[NT][2];  // z: -m, 0 while nothing is seen
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      z[n][0] = z[n][1] = l[n][0] = l[n][1] = 0.0f;
    }
    int get = 0;
    for (int i = 4 * s_begin + warp; i < i_end; i += kWarps) {
      const int first = 16 * keys.chunk(i);
      const bool now = there >> get & 1u;
      const uint8_t* stage = ring + get * F::STAGE;
      get = (get + 1) % F::STAGES;
      copies_wait<F::STAGES - 2>();
      __syncwarp();  // every lane's copies are there, and the stage before is read
      copy();
      if (!now) continue;
      RawKeys<DP> rk;
      RawValues<DP> rv;
      take_keys<DP, FULL>(stage, c.dim, g, q, rk);
      float sc[NT][4] = {};
#pragma unroll
      for (int x = 0; x < F::KW; ++x) {
        uint32_t y[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          codes8(rk.w[t][x], y[t]);
          const uint32_t byte = rk.s[t] >> (8 * (x / 2)) & 0xFFu;
          const uint32_t z = scales2(byte * 0x101u);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[t][e] = h2_mul(y[t][e], z);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 z;
          if constexpr (F::Q_SHARED)
            z = qs[(x * NT + n) * 32 + lane];
          else
            z = make_uint4(qf[n][4 * x], qf[n][4 * x + 1], qf[n][4 * x + 2], qf[n][4 * x + 3]);
          mma(sc[n], y[0][0], y[1][0], y[0][1], y[1][1], z.x, z.y);
          mma(sc[n], y[0][2], y[1][2], y[0][3], y[1][3], z.z, z.w);
        }
      }
      take_values<DP, FULL>(stage, c.dim, g, q, rv);
      if (!keys.all_visible(first)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[n][e] = visible(a, seq, p[n][e & 1], first + g + 8 * (e / 2)) ? sc[n][e] : -INFINITY;
        // what lies behind the end is no number: its weight is 0, and so is its scale
#pragma unroll
        for (int t = 0; t < 4; ++t) rv.s[t] = first + 8 * (t / 2) + 2 * q + t % 2 < seq.length ? rv.s[t] : 0;
      }
      // scores are rounded before the maximum is taken off (not in one step with it): what is left of them
      // is then kMoves at most, whatever their size
      bool up = false;
      float x[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = __fmul_rn(sc[n][e], f[n][e & 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[n][e] = fmaxf(sc[n][e], sc[n][2 + e]);
          up |= x[n][e] - m[n][e] > kMoves;
        }
      }
      if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float d[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = x[n][e];
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
            top = fmaxf(top - kLift, m[n][e]);
            d[e] = top == m[n][e] ? 1.0f : layer::ex2(m[n][e] - top);
            m[n][e] = top;
            z[n][e] = top == -INFINITY ? 0.0f : -top;
            l[n][e] *= d[e];
          }
#pragma unroll
          for (int y = 0; y < F::VN / 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[y][n][e] *= d[e & 1];
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = layer::ex2(__fadd_rn(sc[n][e], z[n][e & 1]));
        l[n][0] += sc[n][0] + sc[n][2];
        l[n][1] += sc[n][1] + sc[n][3];
        pf[n][0] = turned(pack_h2(sc[n][0], sc[n][1]));
        pf[n][1] = turned(pack_h2(sc[n][2], sc[n][3]));
      }
      // values: the codes of two keys side by side in each byte
#pragma unroll
      for (int y = 0; y < F::VW; ++y) {
        const int sh = 8 * (y / 2);
        const uint32_t fa = scales2((rv.s[0] >> sh & 0xFFu) | (rv.s[1] >> sh & 0xFFu) << 8);
        const uint32_t fb = scales2((rv.s[2] >> sh & 0xFFu) | (rv.s[3] >> sh & 0xFFu) << 8);
        const uint32_t a0 = rv.w[0][y], a1 = rv.w[1][y], b0 = rv.w[2][y], b1 = rv.w[3][y];
        uint32_t even_a[4], odd_a[4], even_b[4], odd_b[4];
        codes8((a0 & 0x0F0F0F0Fu) | (a1 << 4 & 0xF0F0F0F0u), even_a);
        codes8((a0 >> 4 & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u), odd_a);
        codes8((b0 & 0x0F0F0F0Fu) | (b1 << 4 & 0xF0F0F0F0u), even_b);
        codes8((b0 >> 4 & 0x0F0F0F0Fu) | (b1 & 0xF0F0F0F0u), odd_b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t v0 = h2_mul(even_a[e], fa), v1 = h2_mul(odd_a[e], fa), v2 = h2_mul(even_b[e], fb),
                         v3 = h2_mul(odd_b[e], fb);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(o[4 * y + e][n], v0, v1, v2, v3, pf[n][0], pf[n][1]);
        }
      }
    }
    copies_wait<0>();

    // the four warps' parts
    __syncthreads();  // the rings are read
    float* mine = os + warp * ROWS * F::O_ROW;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
        const int row = 8 * n + 2 * q + e;
        if (g == 0) {
          ms[warp * ROWS + row] = m[n][e];
          ls[warp * ROWS + row] = sum;
        }
#pragma unroll
        for (int y = 0; y < F::VN / 2; ++y)
          *reinterpret_cast<float2*>(mine + row * F::O_ROW + g * F::VN + 2 * y) = make_float2(o[y][n][e], o[y][n][2 + e]);
      }
    __syncthreads();
    const bool whole = s_begin == 0 && s_end == keys.steps();
    const int slot = 2 * blockIdx.x + (s_begin == 0 ? 1 : 0);  // begun here, or begun before
    float* part = a.ws + F::HEADS + (int64_t)slot * F::SLOT;
    // a thread for each row: what its warps' parts count
    if (threadIdx.x < rows) {
      const int row = threadIdx.x;
      float mi[kWarps], top = -INFINITY, total = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, mi[i] = ms[i * ROWS + row]);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        mi[i] = mi[i] == top ? 1.0f : layer::ex2(mi[i] - top);
        total = fmaf(ls[i * ROWS + row], mi[i], total);
      }
      float share = 1.0f;
      if (whole) {
        const int64_t t = (int64_t)seq.first + (ROWS * r + row) / a.group;
        if (a.lse) a.lse[t * a.Hq + h * a.group + (ROWS * r + row) % a.group] = row_lse(top, total);
        share = total != 0.0f ? alpha_v / total : 0.0f;  // nothing seen: zeros
      } else {
        part[ROWS * DP + row] = top;
        part[ROWS * DP + ROWS + row] = total;
      }
#pragma unroll
      for (int i = 0; i < kWarps; ++i) ms[i * ROWS + row] = mi[i] * share;
    }
    __syncthreads();
    // two values at a time
    for (int x = threadIdx.x; x < rows * (c.dim / 2); x += kThreadsFew) {
      const int row = x / (c.dim / 2), d = 2 * (x - row * (c.dim / 2));
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float2 y = *reinterpret_cast<const float2*>(os + (i * ROWS + row) * F::O_ROW + d);
        const float z = ms[i * ROWS + row];
        sum.x = fmaf(y.x, z, sum.x);
        sum.y = fmaf(y.y, z, sum.y);
      }
      if (whole) {
        const int at = ROWS * r + row, t = at / a.group;
        bf16* out = static_cast<bf16*>(a.o.p) + ((int64_t)seq.first + t) * a.o.ts + (int64_t)(h * a.group + at - t * a.group) * a.o.hs + d;
        if (o_pairs) {
          *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(sum.x, sum.y);
        } else {
          out[0] = layer::from_f32<bf16>(sum.x);
          out[1] = layer::from_f32<bf16>(sum.y);
        }
      } else {
        *reinterpret_cast<float2*>(part + row * DP + d) = sum;
      }
    }
    if (!whole && s_begin == 0 && threadIdx.x == 0)
      heads[blockIdx.x] = {pieces.holds(u1 - 1), seq.first, h, ROWS * r, rows};
    w = u0 + s_end;
  }
}

// The pieces of each unit that is cut, added in order: block i takes the unit that begins in
// piece i and does not end there, a thread four values of one of its rows.
template <int DP, int NT>
__global__ void __launch_bounds__(DP / 4 * 8 * NT) few_join_kernel(AttendArgs a) {
  using F = Few<DP, NT>;
  after_previous();
  const FewHead head = reinterpret_cast<const FewHead*>(a.ws)[blockIdx.x];
  const int row = threadIdx.x / (DP / 4), d = threadIdx.x % (DP / 4) * 4;
  if (head.last < 0 || row >= head.rows || d >= a.c.dim) return;
  const float* p = a.ws + F::HEADS + (2 * (int64_t)blockIdx.x + 1) * F::SLOT;
  float top = p[F::ROWS * DP + row], l = p[F::ROWS * DP + F::ROWS + row];
  float4 sum = *reinterpret_cast<const float4*>(p + row * DP + d);
#pragma unroll 4
  for (int j = blockIdx.x + 1; j <= head.last; ++j) {
    const float* x = a.ws + F::HEADS + 2 * (int64_t)j * F::SLOT;
    const float mj = x[F::ROWS * DP + row], lj = x[F::ROWS * DP + F::ROWS + row];
    const float4 oj = *reinterpret_cast<const float4*>(x + row * DP + d);
    const float next = fmaxf(top, mj);
    const float f = top == next ? 1.0f : layer::ex2(top - next), fj = mj == next ? 1.0f : layer::ex2(mj - next);
    sum.x = fmaf(oj.x, fj, sum.x * f);
    sum.y = fmaf(oj.y, fj, sum.y * f);
    sum.z = fmaf(oj.z, fj, sum.z * f);
    sum.w = fmaf(oj.w, fj, sum.w * f);
    l = fmaf(lj, fj, l * f);
    top = next;
  }
  const int at = head.row + row;
  const int64_t t = (int64_t)head.first + at / a.group;
  const int h = head.head * a.group + at % a.group;
  const float share = l != 0.0f ? a.c.alpha[1] / l : 0.0f;  // nothing seen: zeros
  bf16* out = static_cast<bf16*>(a.o.p) + t * a.o.ts + (int64_t)h * a.o.hs + d;
  const float v[4] = {sum.x * share, sum.y * share, sum.z * share, sum.w * share};
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = layer::from_f32<bf16>(v[e]);
  if (d == 0 && a.lse) a.lse[t * a.Hq + h] = row_lse(top, l);
}

template <int DP, int NT, bool FULL>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  using F = Few<DP, NT>;
  cudaError_t e = cudaFuncSetAttribute(few_kernel<DP, NT, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_early(few_kernel<DP, NT, FULL>, dim3((unsigned)F::BLOCKS), kThreadsFew, F::SMEM, s, a);
  if (e != cudaSuccess) return e;
  return launch_early(few_join_kernel<DP, NT>, dim3((unsigned)F::BLOCKS), DP / 4 * F::ROWS, 0, s, a);
}
template <int DP, int NT>
cudaError_t by_dim(const AttendArgs& a, cudaStream_t s) {
  return a.c.dim == DP ? launch<DP, NT, true>(a, s) : launch<DP, NT, false>(a, s);
}

// Tiles of 8 rows if an average sequence's fit one, else of 16.  (Sixteen sequences of 20 rows in a
// window of 2048: one tile of 24 rows, which takes so many registers that an SM holds 8 warps, 52 us;
// two of 16 45.)
static int tiles_of(int64_t T, int group, int64_t sequences) {
  return (T + sequences - 1) / sequences * group <= 8 ? 1 : 2;
}

}  // namespace attention

int64_t attend_few_workspace(int64_t T, int group, int dim, int64_t sequences) {
  using namespace attention;
  const int n = tiles_of(T, group, sequences);
  const int64_t floats = dim <= 64    ? (n == 1 ? Few<64, 1>::FLOATS : Few<64, 2>::FLOATS)
                         : dim <= 128 ? (n == 1 ? Few<128, 1>::FLOATS : Few<128, 2>::FLOATS)
                                      : (n == 1 ? Few<256, 1>::FLOATS : Few<256, 2>::FLOATS);
  return floats * (int64_t)sizeof(float);
}

cudaError_t launch_attend_few(const AttendArgs& a, cudaStream_t s) {
  using namespace attention;
  const int n = tiles_of(a.c.T, a.group, a.c.sequences);
  if (a.c.dim <= 64) return n == 1 ? by_dim<64, 1>(a, s) : by_dim<64, 2>(a, s);
  if (a.c.dim <= 128) return n == 1 ? by_dim<128, 1>(a, s) : by_dim<128, 2>(a, s);
  return n == 1 ? by_dim<256, 1>(a, s) : by_dim<256, 2>(a, s);
}

}  // namespace nvfp4
