/*
 * nvfp4_attention.h -- C ABI of the attention operators on an NVFP4 cache: the norm
 * and rotation of queries and keys and its gradient, a paged cache of keys and
 * values in 4 bits (write and read), and the attention that reads it, for prompts
 * and for single tokens.  Built for GB300 (sm_103a) into libnvfp4_attention.so;
 * status values and nvfp4_strerror are those of nvfp4.h (libnvfp4.so).
 *
 * Between the two linear layers of an attention block:
 *   nvfp4_linear (queries, keys, values) -> nvfp4_qk_rope -> nvfp4_cache_write ->
 *   nvfp4_cache_attention -> nvfp4_quantize -> nvfp4_linear (residual).
 *
 * Conventions, as in nvfp4_layer.h: pointers named *_dev, and those inside the two
 * structs below, are device pointers owned by the caller; the library allocates
 * nothing and keeps nothing between calls but what its kernels' launches need on a
 * device; several host threads may call it at once; every call is asynchronous on
 * `stream` (a cudaStream_t as void*, NULL = legacy default stream); argument errors
 * are returned at once, before anything is enqueued.  An "is_bf16" argument is 1 for
 * bf16 elements and 0 for fp32.  Arithmetic is fp32 but where a call says otherwise;
 * a bf16 result is rounded once, to nearest even.  The results do not depend on the
 * order in which blocks run: the same call on the same device gives the same bits.
 * Workspaces as in nvfp4_layer.h: scratch memory, 16-byte aligned, of at least the
 * bytes that the matching *_workspace function returns on the same device, not
 * shared by calls that may run at the same time; needed and NULL is ERR_NULL, too
 * small ERR_SHAPE.  Outputs must not overlap inputs, except where a call says that
 * they may.
 *
 * Token tensors (T tokens x H heads x D values) have D contiguous and any stride, in
 * elements, from token to token and from head to head (0 <= stride, and at most 2^58 from the
 * first to the last); outputs must not overlap themselves.  Any base address aligned to the element is accepted;
 * heads that begin at 16 bytes are faster.
 */
#ifndef NVFP4_ATTENTION_H
#define NVFP4_ATTENTION_H

#include <stdint.h>

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A token tensor (the pointer's type is given by the call). */
typedef struct {
  void* data;
  int64_t token_stride, head_stride; /* in elements */
} nvfp4_tokens;

/*
 * A paged cache of keys and values.  Row r of page p of key/value head h holds one
 * token: `dim` values as E2M1 codes (dim/2 bytes, the first value of a pair in the low
 * nibble) and one E4M3 scale for each 16 of them (dim/16 bytes), at
 *   codes  + p * code_page  + h * code_head  + r * code_row
 *   scales + p * scale_page + h * scale_head + r * scale_row     (strides in bytes),
 * the same strides for keys and for values.  A value is code * scale * alpha, with
 * alpha_dev[0] for keys and alpha_dev[1] for values.  The scales within a sequence's
 * length are finite (as nvfp4_cache_write leaves them); what lies behind it is not used.
 *   dim        a multiple of 32, 32..256
 *   page_size  a multiple of 16, 16..65536
 *   pages      0..2^31 - 1;  heads 1..65535
 *   codes and their strides: multiples of 16 bytes; scales and theirs: of 2 bytes;
 *   no stride may be less than what it steps over makes necessary for rows not to
 *   overlap: any order of page, head and row is accepted; strides of pages and rows are
 *   below 2^32, those of heads at most 2^45.
 */
typedef struct {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const float* alpha_dev; /* float[2] */
  int64_t pages;
  int heads, page_size, dim;
  int64_t code_page, code_head, code_row;
  int64_t scale_page, scale_head, scale_row;
} nvfp4_kv_cache;

/*
 * Which tokens a call is on.  Sequence b holds lengths[b] tokens in the cache; the
 * call's rows starts[b] .. starts[b+1] - 1 are its last n = starts[b+1] - starts[b]
 * ones: row starts[b] + i is at position lengths[b] - n + i.  Position j lies in row
 * j % page_size of page table[b * table_stride + j / page_size].
 *   starts   int32[sequences + 1], not decreasing, within 0..T
 *   lengths  int32[sequences], within 0..table_width * page_size
 *   table    page numbers within 0..pages - 1 where positions below lengths[b] use them
 * Sequences whose starts or length are out of range are left out, their rows left as
 * they are; a token whose page number is out of range is left out by itself.  Either
 * sets *status_dev (int, or NULL) to NVFP4_ERR_INDEX; it is untouched otherwise (the
 * caller zeroes it).  Rows before starts[0] and from starts[sequences] on are left as
 * they are.
 */
typedef struct {
  const int32_t *starts, *lengths, *table;
  int64_t sequences, table_width, table_stride;
} nvfp4_batch;

/*
 * nvfp4_qk_rope -- norm of each head's queries and keys, and their rotation, in one
 * pass.  For each token and head
 *   y = x * rsqrt(sum(x^2)/D + eps) * gamma      (without norm: y = x),
 * then pair i of the first 2 * rotated values is turned by the angle
 * positions[t] * inv_freq[i]:  (a, b) -> (a cos - b sin, b cos + a sin).  Pair i is
 * values (i, i + rotated), or (2i, 2i + 1) with interleaved = 1; the other values pass.
 * The angle is the product of the two numbers as they are, reduced in 64 bits: far
 * positions lose nothing (off by |position| max(1, |inv_freq|) 2^-53 turns).
 *
 *   q, k          T x q_heads x D and T x k_heads x D, x's type;  heads 0..65535
 *   D             a multiple of 2, 2..512;  rotated 0..D/2 (number of pairs)
 *   positions_dev int32[T];  inv_freq_dev  float[rotated], finite
 *   norm          1 or 0;  eps finite and >= 0 (used with norm)
 *   gamma_q_dev, gamma_k_dev  D weights or NULL (ones), fp32 (w_is_bf16 = 0) or bf16;
 *                 both NULL without norm
 *   out_q, out_k  as q and k, y's type; may be q and k themselves (same type and strides)
 * A NaN or Inf in a head of a token touches no other, and without the norm no other pair or
 * passing value; the sum of squares of a head is formed in fp32 and has to stay finite (and
 * above 0 where eps is 0).
 * Errors: SHAPE, NULL, ALIGN, FLAGS (eps, gammas without norm), CUDA.
 */
NVFP4_API int nvfp4_qk_rope(const nvfp4_tokens* q, const nvfp4_tokens* k, int x_is_bf16, int64_t T, int q_heads,
                            int k_heads, int D, int rotated, int interleaved, const int32_t* positions_dev,
                            const float* inv_freq_dev, int norm, float eps, const void* gamma_q_dev,
                            const void* gamma_k_dev, int w_is_bf16, const nvfp4_tokens* out_q,
                            const nvfp4_tokens* out_k, int y_is_bf16, void* stream);

/*
 * nvfp4_qk_rope_backward -- its gradient.  With g = dy turned back by the same angles,
 * xhat = x * r and r = rsqrt(sum(x^2)/D + eps), per head
 *   dx = r * (g gamma - xhat * sum(g gamma xhat)/D)      (without norm: dx = g),
 * and over tokens and heads dgamma = sum(g * xhat).
 *
 *   dq, dk        gradients of out_q and out_k, dy's type
 *   q, k          the forward pass's inputs (not read without norm: may be NULL)
 *   dx_q, dx_k    of x's type; may be dq and dk themselves, or q and k (same type and
 *                 strides)
 *   dgamma_q_dev, dgamma_k_dev  D floats each or NULL; overwritten; NULL without norm
 *   workspace_dev nvfp4_qk_rope_backward_workspace(T, q_heads, k_heads, D) bytes, needed
 *                 where a dgamma is wanted
 * The sums over tokens are formed in a fixed order.
 * Errors: SHAPE, NULL, ALIGN, FLAGS, CUDA.
 */
NVFP4_API int64_t nvfp4_qk_rope_backward_workspace(int64_t T, int q_heads, int k_heads, int D);
NVFP4_API int nvfp4_qk_rope_backward(const nvfp4_tokens* dq, const nvfp4_tokens* dk, int dy_is_bf16,
                                     const nvfp4_tokens* q, const nvfp4_tokens* k, int x_is_bf16, int64_t T,
                                     int q_heads, int k_heads, int D, int rotated, int interleaved,
                                     const int32_t* positions_dev, const float* inv_freq_dev, int norm, float eps,
                                     const void* gamma_q_dev, const void* gamma_k_dev, int w_is_bf16,
                                     const nvfp4_tokens* dx_q, const nvfp4_tokens* dx_k, float* dgamma_q_dev,
                                     float* dgamma_k_dev, void* workspace_dev, int64_t workspace_bytes, void* stream);

/*
 * nvfp4_cache_write -- the batch's keys and values into the cache.  For each block of
 * 16 values x of a head, with b = max |x|,
 *   scale = E4M3(b / (6 alpha)), code = E2M1(x / (scale alpha)),
 * quotients and roundings to nearest even, saturating; a block whose scale is 0 has
 * signed zeros as codes.  Where alpha is a power of two nothing but these two
 * roundings comes between x and the code.  (nvfp4_quantize multiplies by the reciprocal instead,
 * which may differ for x next to the middle of two codes.)
 *
 *   k, v        T x heads x dim, bf16 or fp32
 *   status_dev  int or NULL: NVFP4_ERR_NONFINITE if a value is NaN (stored as 0) or
 *               infinite (stored as the largest code, beside a saturated scale), so that
 *               no later product with the cache meets one; NVFP4_ERR_RANGE if an alpha
 *               is not within 2^-100..2^100 (nothing is written then); NVFP4_ERR_INDEX
 *               as for every batch, and for a row whose position is negative
 *               (starts[b+1] - starts[b] > lengths[b]), which is left out.  Several: one
 *               of them.
 * Two rows of one call must not lie in the same place (a page that two sequences, or
 * one sequence twice, name for new tokens): that place's contents are then a mixture.
 * Errors: SHAPE, NULL, ALIGN, CUDA.
 */
NVFP4_API int nvfp4_cache_write(const nvfp4_tokens* k, const nvfp4_tokens* v, int x_is_bf16, int64_t T,
                                const nvfp4_kv_cache* cache, const nvfp4_batch* batch, int* status_dev, void* stream);

/*
 * nvfp4_cache_read -- the batch's keys and values out of the cache: code * scale * alpha,
 * rounded to y's type.  A row whose page number is out of range or whose position is
 * negative becomes zeros (and sets *status_dev).
 *
 *   k, v  T x heads x dim, bf16 or fp32; either's data may be NULL (not wanted)
 * Errors: SHAPE, NULL, ALIGN, CUDA.
 */
NVFP4_API int nvfp4_cache_read(const nvfp4_tokens* k, const nvfp4_tokens* v, int y_is_bf16, int64_t T,
                               const nvfp4_kv_cache* cache, const nvfp4_batch* batch, int* status_dev, void* stream);

/*
 * nvfp4_cache_attention -- the batch's queries attend to the cache.  Query head h reads
 * key/value head h / (q_heads / heads).  With position p of a row,
 *   s_j = scale * (q . k_j) over the visible keys j,  lse = log(sum exp(s_j)),
 *   o = sum exp(s_j - lse) v_j.
 * causal = 1: key j is visible if j <= p and, with window > 0, p - j < window or
 * j < sinks.  causal = 0: all lengths[b] keys are visible (window and sinks must be 0).
 * A row that sees no key (a negative position, a length of 0, pages out of range)
 * becomes zeros, its lse -Inf.
 *
 *   q         T x q_heads x dim, bf16;  q_heads a multiple of heads, at most 65535
 *   o         as q;  may be q itself (same strides)
 *   lse_dev   T x q_heads floats (natural logarithm) or NULL
 *   scale     finite; scale * alpha, and that times a row's largest query, stay finite in fp32
 *   window    0 (no window) .. 2^31 - 1;  sinks 0 .. 2^31 - 1, 0 without a window
 *   workspace_dev  nvfp4_cache_attention_workspace(T, q_heads, heads, dim, sequences) bytes
 * The products take bf16 queries (scaled by a power of two per row into fp16: exactly down
 * to 2^-31 of the row's largest, within 2^-39 of it below) and the cache's values exactly;
 * sums are fp32.  A weight is rounded to fp16 where it meets the values (half a step: 2^-11
 * of the weight, or 2^-32 of the row's largest weight where that is more), not where it is
 * summed.
 * NaN or Inf in a query makes that row NaN (or whatever their formula gives) and touches no other.
 * Errors: SHAPE, NULL, ALIGN, FLAGS (scale; window or sinks without causal; sinks without
 * a window; negative ones), CUDA.
 */
NVFP4_API int64_t nvfp4_cache_attention_workspace(int64_t T, int q_heads, int heads, int dim, int64_t sequences);
NVFP4_API int nvfp4_cache_attention(const nvfp4_tokens* q, int64_t T, int q_heads, const nvfp4_kv_cache* cache,
                                    const nvfp4_batch* batch, float scale, int causal, int64_t window, int64_t sinks,
                                    const nvfp4_tokens* o, float* lse_dev, void* workspace_dev,
                                    int64_t workspace_bytes, int* status_dev, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_ATTENTION_H */
