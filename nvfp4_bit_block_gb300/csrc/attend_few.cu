// attend_few.cu -- attention of sequences with few new rows (tokens times the query heads
// that share a key head) to the NVFP4 cache: the next token, or a few drafted ones.
//
// The cache's bytes are the floor: 9/16 byte per value, read once for all heads of a group.
// A unit of work is 16 rows of one key head; its visible keys are cut into steps of 64 and the
// steps of all units form one line that is cut into equal pieces, one per block, so that one
// long sequence and many short ones fill the GPU alike.  Pieces that are part of a unit leave
// (m, l, o) in the workspace and a second kernel joins them in order.
//
// Within a step each of a block's four warps takes 16 keys, all the way from the cache's bytes
// to the output in registers: S = Q K^T and O += P V as m16n8k16 products in fp16 with fp32
// sums.  A code times its scale has at most 6 significant bits within 2^-10..2688, so it is
// exact in fp16; queries are scaled by a power of two per row.  Which of a product's k's (and of
// the output's columns) a value counts as is free, as long as both operands agree: each lane
// loads bytes that lie side by side and uses them where they are.  Lane (g, c) = (lane / 4,
// lane % 4) has for key rows g and 8 + g the c-th quarter of the values, and for the value rows
// 2c, 2c + 1, 8 + 2c, 9 + 2c the g-th eighth.
//
// The running maximum moves only where a score passes it by more than 2^8: weights stay below
// 256, where fp16 holds them as well as below 1, and most steps leave o alone.
#include <cmath>

#include "attend.cuh"

namespace nvfp4 {
namespace attention {

constexpr int kWarps = 4;
constexpr int kThreadsFew = 32 * kWarps;

template <int DP>
struct Few {
  static constexpr int KW = DP / 32;    // words of a lane's part of a key (DP / 4 values)
  static constexpr int KS = DP / 64;    // its scales
  static constexpr int STEPS = DP / 16; // products over a key
  static constexpr int VN = DP / 8;     // values of a lane's part of a value row
  static constexpr int VW = VN / 8;     // words of it
  static constexpr int VS = VN >= 32 ? 2 : 1;
  // A row of o in shared memory: value n * VN + i at 9 i + n; rows 8 banks apart.
  static constexpr int ROW = DP == 64 ? 72 : DP == 128 ? 168 : 296;
  static constexpr int QBYTES = DP == 256 ? STEPS * 32 * 16 : 0;
  static constexpr int SMEM = kWarps * 16 * ROW * 4 + 2 * kWarps * 16 * 4 + QBYTES;
};

// One lane's bytes of 16 keys and values.
template <int DP>
struct Raw {
  uint32_t k[2][Few<DP>::KW], v[4][Few<DP>::VW];
  uint32_t ks[2], vs[4];  // scale bytes, first lowest
};

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes of the chunk at `page`, row `row` (a multiple of 16); parts beyond D are zeros.
template <int DP>
__device__ __forceinline__ void load_chunk(const CacheView& c, int h, int page, int row, Raw<DP>& r) {
  using F = Few<DP>;
  const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int64_t co = (int64_t)page * c.cp + (int64_t)h * c.ch, so = (int64_t)page * c.sp + (int64_t)h * c.sh;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t at = row + 8 * t + g;
    const uint8_t* p = c.kc + co + at * c.cr + q * (DP / 8);
    const uint8_t* s = c.ks + so + at * c.sr + q * F::KS;
    if constexpr (DP == 64) {
      const bool on = q * 16 < c.dim;
      const uint2 w = on ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
      r.k[t][0] = w.x;
      r.k[t][1] = w.y;
      r.ks[t] = on ? *s : 0;
    } else {
      r.ks[t] = 0;
#pragma unroll
      for (int i = 0; i < F::KW / 4; ++i) {
        const bool on = q * (DP / 4) + 32 * i < c.dim;
        const uint4 w = on ? *reinterpret_cast<const uint4*>(p + 16 * i) : make_uint4(0, 0, 0, 0);
        r.k[t][4 * i] = w.x;
        r.k[t][4 * i + 1] = w.y;
        r.k[t][4 * i + 2] = w.z;
        r.k[t][4 * i + 3] = w.w;
        if (on) r.ks[t] |= (uint32_t)*reinterpret_cast<const uint16_t*>(s + 2 * i) << (16 * i);
      }
    }
  }
  const bool on = g * F::VN < c.dim;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t at = row + 8 * (t / 2) + 2 * q + t % 2;
    const uint8_t* p = c.vc + co + at * c.cr + g * (DP / 16);
    const uint8_t* s = c.vs + so + at * c.sr + g * F::VN / 16;
    r.vs[t] = 0;
    if constexpr (DP == 64) {
      r.v[t][0] = on ? *reinterpret_cast<const uint32_t*>(p) : 0;
      if (on) r.vs[t] = *s;
    } else if constexpr (DP == 128) {
      const uint2 w = on ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
      r.v[t][0] = w.x;
      r.v[t][1] = w.y;
      if (on) r.vs[t] = *s;
    } else {
      const uint4 w = on ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
      r.v[t][0] = w.x;
      r.v[t][1] = w.y;
      r.v[t][2] = w.z;
      r.v[t][3] = w.w;
      if (on) r.vs[t] = *reinterpret_cast<const uint16_t*>(s);
    }
  }
}

// A lane's part of a row's queries in fp16; returns what undoes their scaling.
template <int DP>
__device__ __forceinline__ float load_query(const AttendArgs& a, bool vec, bool on, int64_t token, int head, uint32_t* h) {
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
  const float down = query_down(top);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) h[i] = pack_h2(bf16_lo(h[i]) * down, bf16_hi(h[i]) * down);
  return query_up(top);
}

template <int DP>
__global__ void __launch_bounds__(kThreadsFew, few_per_sm(DP)) few_kernel(AttendArgs a) {
  using F = Few<DP>;
  extern __shared__ __align__(16) float sm[];
  __shared__ Line line;
  const CacheView& c = a.c;
  after_previous();
  if (blockIdx.x == 0) check_batch(c);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, q = lane % 4;
  float* os = sm;                                // [warps][16][ROW]
  float* ms = sm + kWarps * 16 * F::ROW;         // [warps][16]
  float* ls = ms + kWarps * 16;                  // [warps][16]
  uint4* qs = reinterpret_cast<uint4*>(ls + kWarps * 16);  // [STEPS][32], DP = 256 only

  find_line<kThreadsFew>(
      c, line, [&](int b) {
        Sequence s;
        load_few(a, b, s);
        return sequence_steps(a, s) * c.heads;
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
  const float alpha_v = c.alpha[1], scale = a.scale * c.alpha[0] * layer::kLog2e;

  const bool vec = rows_at_16(a.q);

  while (w < w_end) {
    // the unit that w is in
    int64_t per_head = sequence_steps(a, seq);
    while (w >= base + per_head * c.heads) {
      base += per_head * c.heads;
      load_few(a, ++b, seq);
      per_head = sequence_steps(a, seq);
    }
    const int h = (int)((w - base) / per_head);
    int64_t u0 = base + h * per_head;
    int r = 0;
    Keys<16> keys = tile_keys(a, seq, 0);
    while (w >= u0 + keys.steps()) {
      u0 += keys.steps();
      keys = tile_keys(a, seq, ++r);
    }
    const int64_t u1 = u0 + keys.steps();
    const int s_begin = (int)(w - u0), s_end = (int)((w_end < u1 ? w_end : u1) - u0);
    const int rows = min(16, seq.rows * a.group - 16 * r);

    // queries
    const int row0 = 16 * r + g, row1 = row0 + 8;
    const bool on0 = g < rows, on1 = g + 8 < rows;
    const int t0 = on0 ? row0 / a.group : 0, t1 = on1 ? row1 / a.group : 0;
    uint32_t qf[F::STEPS][4];
    float f0, f1;
    {
      uint32_t x[F::STEPS * 2];
      f0 = scale * load_query<DP>(a, vec, on0, (int64_t)seq.first + t0, h * a.group + (on0 ? row0 % a.group : 0), x);
#pragma unroll
      for (int j = 0; j < F::STEPS; ++j) {
        qf[j][0] = x[2 * j];
        qf[j][2] = x[2 * j + 1];
      }
      f1 = scale * load_query<DP>(a, vec, on1, (int64_t)seq.first + t1, h * a.group + (on1 ? row1 % a.group : 0), x);
#pragma unroll
      for (int j = 0; j < F::STEPS; ++j) {
        qf[j][1] = x[2 * j];
        qf[j][3] = x[2 * j + 1];
      }
    }
    if constexpr (DP == 256) {
      __syncthreads();
      if (warp == 0)
#pragma unroll
        for (int j = 0; j < F::STEPS; ++j) qs[j * 32 + lane] = make_uint4(qf[j][0], qf[j][1], qf[j][2], qf[j][3]);
      __syncthreads();
    }
    const int p0 = seq.length - seq.rows + t0, p1 = seq.length - seq.rows + t1;

    float o[F::VN][4] = {};
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    Raw<DP> next;
    int next_chunk = -1, next_page = -1;
    auto fetch = [&](int s) {
      const int i = 4 * s + warp;
      next_page = -1;
      next_chunk = -1;
      if (s >= s_end || i >= keys.count) return;
      next_chunk = keys.chunk(i);
      next_page = page_of(c, b, 16 * next_chunk);
      if (next_page >= 0)
        load_chunk<DP>(c, h, next_page, 16 * next_chunk % c.page_size, next);
      else
        set_status(c.status, NVFP4_ERR_INDEX);
    };
    fetch(s_begin);
    for (int s = s_begin; s < s_end; ++s) {
      Raw<DP> raw = next;
      const int first = 16 * next_chunk, page = next_page;
      const bool there = next_chunk >= 0 && page >= 0;
      fetch(s + 1);
      if (!there) continue;
      // scores
      float sc[2][4] = {};
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < F::KW; ++i) {
          uint32_t x[4];
          codes8(raw.k[t][i], x);
          const uint32_t byte = raw.ks[t] >> (8 * (i / 2)) & 0xFFu;
          const uint32_t f = scales2(byte | byte << 8);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 2 * i + e;
            if constexpr (DP == 256) {
              const uint4 y = qs[j * 32 + lane];
              const uint32_t qa[4] = {y.x, y.y, y.z, y.w};
              mma(sc[t], qa, h2_mul(x[2 * e], f), h2_mul(x[2 * e + 1], f));
            } else {
              mma(sc[t], qf[j], h2_mul(x[2 * e], f), h2_mul(x[2 * e + 1], f));
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[t][0] *= f0;
        sc[t][1] *= f0;
        sc[t][2] *= f1;
        sc[t][3] *= f1;
      }
      if (!keys.all_visible(first)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = first + 8 * t + 2 * q + e;
            if (!visible(a, seq, p0, j)) sc[t][e] = -INFINITY;
            if (!visible(a, seq, p1, j)) sc[t][2 + e] = -INFINITY;
          }
        // what lies behind the end is no number: its weight is 0, and so is its scale
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (first + 8 * (t / 2) + 2 * q + t % 2 >= seq.length) raw.vs[t] = 0;
      }
      const float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      const float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      if (__any_sync(0xFFFFFFFFu, x0 > m0 + 8.0f || x1 > m1 + 8.0f)) {
        float n0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1)), n1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 1));
        n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, 2)));
        n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, 2)));
        const float d0 = n0 == m0 ? 1.0f : layer::ex2(m0 - n0), d1 = n1 == m1 ? 1.0f : layer::ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= d0;
        l1 *= d1;
#pragma unroll
        for (int i = 0; i < F::VN; ++i) {
          o[i][0] *= d0;
          o[i][1] *= d0;
          o[i][2] *= d1;
          o[i][3] *= d1;
        }
      }
      const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[t][0] = layer::ex2(sc[t][0] - z0);
        sc[t][1] = layer::ex2(sc[t][1] - z0);
        sc[t][2] = layer::ex2(sc[t][2] - z1);
        sc[t][3] = layer::ex2(sc[t][3] - z1);
      }
      l0 += (sc[0][0] + sc[0][1]) + (sc[1][0] + sc[1][1]);
      l1 += (sc[0][2] + sc[0][3]) + (sc[1][2] + sc[1][3]);
      const uint32_t pf[4] = {pack_h2(sc[0][0], sc[0][1]), pack_h2(sc[0][2], sc[0][3]), pack_h2(sc[1][0], sc[1][1]),
                              pack_h2(sc[1][2], sc[1][3])};
      // values: the codes of two keys side by side in each byte
#pragma unroll
      for (int i = 0; i < F::VW; ++i) {
        const int sh = 8 * (i / 2);
        const uint32_t fa = scales2((raw.vs[0] >> sh & 0xFFu) | (raw.vs[1] >> sh & 0xFFu) << 8);
        const uint32_t fb = scales2((raw.vs[2] >> sh & 0xFFu) | (raw.vs[3] >> sh & 0xFFu) << 8);
        const uint32_t a0 = raw.v[0][i], a1 = raw.v[1][i], b0 = raw.v[2][i], b1 = raw.v[3][i];
        uint32_t even_a[4], odd_a[4], even_b[4], odd_b[4];
        codes8((a0 & 0x0F0F0F0Fu) | (a1 << 4 & 0xF0F0F0F0u), even_a);
        codes8((a0 >> 4 & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u), odd_a);
        codes8((b0 & 0x0F0F0F0Fu) | (b1 << 4 & 0xF0F0F0F0u), even_b);
        codes8((b0 >> 4 & 0x0F0F0F0Fu) | (b1 & 0xF0F0F0F0u), odd_b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mma(o[8 * i + 2 * e], pf, h2_mul(even_a[e], fa), h2_mul(even_b[e], fb));
          mma(o[8 * i + 2 * e + 1], pf, h2_mul(odd_a[e], fa), h2_mul(odd_b[e], fb));
        }
      }
    }

    // the four warps' parts
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, x);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, x);
    }
    __syncthreads();  // the part before is read
    if (q == 0) {
      ms[warp * 16 + g] = m0;
      ms[warp * 16 + 8 + g] = m1;
      ls[warp * 16 + g] = l0;
      ls[warp * 16 + 8 + g] = l1;
    }
    float* mine = os + warp * 16 * F::ROW;
#pragma unroll
    for (int i = 0; i < F::VN; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) mine[(g + 8 * (e / 2)) * F::ROW + 9 * i + 2 * q + e % 2] = o[i][e];
    __syncthreads();
    const bool whole = s_begin == 0 && s_end == keys.steps();
    const int slot = 2 * blockIdx.x + (s_begin == 0 ? 1 : 0);  // begun here, or begun before
    float* part = a.ws + few_head_floats(DP) + (int64_t)slot * few_slot_floats(DP);
    for (int x = threadIdx.x; x < rows * c.dim; x += kThreadsFew) {
      const int row = x / c.dim, d = x % c.dim, at = row * F::ROW + 9 * (d % F::VN) + d / F::VN;
      float top = ms[row];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) top = fmaxf(top, ms[i * 16 + row]);
      float sum = 0.0f, l = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float mi = ms[i * 16 + row], f = mi == top ? 1.0f : layer::ex2(mi - top);
        sum = fmaf(os[i * 16 * F::ROW + at], f, sum);
        l = fmaf(ls[i * 16 + row], f, l);
      }
      if (whole) {
        finish(a, seq, h, 16 * r + row, d, sum, top, l, alpha_v);
      } else {
        part[row * DP + d] = sum;
        if (d == 0) {
          part[16 * DP + row] = top;
          part[16 * DP + 16 + row] = l;
        }
      }
    }
    if (!whole && s_begin == 0 && threadIdx.x == 0)
      heads[blockIdx.x] = {pieces.holds(u1 - 1), seq.first, h, r, rows};
    w = u0 + s_end;
  }
}

// The pieces of each unit that is cut, added in order: block (i, y) takes the unit that begins in
// piece i and does not end there, rows y, y + gridDim.y, ..
template <int DP>
__global__ void __launch_bounds__(DP) few_join_kernel(AttendArgs a) {
  after_previous();
  const FewHead head = reinterpret_cast<const FewHead*>(a.ws)[blockIdx.x];
  if (head.last < 0) return;
  const float* slots = a.ws + few_head_floats(DP);
  const int64_t n = few_slot_floats(DP);
  Sequence seq = {head.first, 0, 0};
  const float alpha_v = a.c.alpha[1];
  const int d = threadIdx.x;
  for (int row = blockIdx.y; row < head.rows; row += gridDim.y) {
    const float* p = slots + (2 * (int64_t)blockIdx.x + 1) * n;
    float top = p[16 * DP + row], l = p[16 * DP + 16 + row], sum = d < a.c.dim ? p[row * DP + d] : 0.0f;
#pragma unroll 4
    for (int j = blockIdx.x + 1; j <= head.last; ++j) {
      const float* x = slots + 2 * (int64_t)j * n;
      const float mj = x[16 * DP + row], lj = x[16 * DP + 16 + row], oj = d < a.c.dim ? x[row * DP + d] : 0.0f;
      const float next = fmaxf(top, mj);
      const float f = top == next ? 1.0f : layer::ex2(top - next), fj = mj == next ? 1.0f : layer::ex2(mj - next);
      sum = fmaf(oj, fj, sum * f);
      l = fmaf(lj, fj, l * f);
      top = next;
    }
    if (d < a.c.dim) finish(a, seq, head.head, 16 * head.tile + row, d, sum, top, l, alpha_v);
  }
}

template <int DP>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  using F = Few<DP>;
  cudaError_t e = cudaFuncSetAttribute(few_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
  if (e != cudaSuccess) return e;
  constexpr int G = few_blocks(DP);
  e = launch_early(few_kernel<DP>, dim3((unsigned)G), kThreadsFew, F::SMEM, s, a);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.c.T * a.group;
  return launch_early(few_join_kernel<DP>, dim3((unsigned)G, (unsigned)(rows < 4 ? rows : 4)), DP, 0, s, a);
}

}  // namespace attention

cudaError_t launch_attend_few(const AttendArgs& a, cudaStream_t s) {
  using namespace attention;
  if (a.c.dim <= 64) return launch<64>(a, s);
  if (a.c.dim <= 128) return launch<128>(a, s);
  return launch<256>(a, s);
}

}  // namespace nvfp4
