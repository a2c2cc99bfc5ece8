// attention_api.cu -- the C ABI declared in include/nvfp4_attention.h: host-side
// argument validation and dispatch.  Nothing here allocates memory or keeps state;
// every call enqueues work on the caller's stream.
#include "nvfp4_attention.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attention_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
uintptr_t elem(int is_bf16) { return is_bf16 ? 2 : 4; }
int launch_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Sizes are bounded so that token and head counts fit 32 bits; offsets are formed in
// 64 bits everywhere, and a stride times what it is stepped over stays far below 2^63.
constexpr int64_t kMaxExtent = (int64_t)1 << 58, kMaxHeadStride = (int64_t)1 << 45;
bool bad_stride(int64_t stride, int64_t n) { return stride < 0 || (n > 1 && stride > kMaxExtent / (n - 1)); }
bool bad_tokens(const nvfp4_tokens* t, int64_t T, int heads) {
  return bad_stride(t->token_stride, T) || bad_stride(t->head_stride, heads);
}
nvfp4::Tokens view(const nvfp4_tokens* t) { return {t->data, t->token_stride, t->head_stride}; }

int zero(void* p, int64_t bytes, cudaStream_t s) {
  return p && bytes ? launch_status(cudaMemsetAsync(p, 0, (size_t)bytes, s)) : NVFP4_OK;
}
int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return NVFP4_OK;
  if (!ws) return NVFP4_ERR_NULL;
  if (have < need) return NVFP4_ERR_SHAPE;
  return aligned(ws, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

bool bad_rope_sizes(int64_t T, int Hq, int Hk, int D, int rotated) {
  return T < 0 || T > INT32_MAX || Hq < 0 || Hk < 0 || Hq > 65535 || Hk > 65535 || D < 2 || D > 512 || D % 2 ||
         rotated < 0 || rotated > D / 2;
}

// What both directions check of their shared arguments.
int check_rope(const nvfp4_tokens* const* t, const uintptr_t* es, int n, int64_t T, int Hq, int Hk, int D, int rotated,
               const int32_t* pos, const float* freq, int norm, float eps, const void* gq, const void* gk, int wb) {
  if (bad_rope_sizes(T, Hq, Hk, D, rotated)) return NVFP4_ERR_SHAPE;
  for (int i = 0; i < n; ++i) {
    if (!t[i]) return NVFP4_ERR_NULL;
    if (bad_tokens(t[i], T, i % 2 ? Hk : Hq)) return NVFP4_ERR_SHAPE;
  }
  if (norm ? (!(eps >= 0.0f) || std::isinf(eps)) : (gq || gk)) return NVFP4_ERR_FLAGS;
  const bool empty = T == 0 || Hq + Hk == 0;
  if (!empty) {
    for (int i = 0; i < n; ++i)
      if (!t[i]->data && (i % 2 ? Hk : Hq) > 0) return NVFP4_ERR_NULL;
    if (rotated > 0 && (!pos || !freq)) return NVFP4_ERR_NULL;
  }
  for (int i = 0; i < n; ++i)
    if (!aligned(t[i]->data, es[i])) return NVFP4_ERR_ALIGN;
  if (!aligned(pos, 4) || !aligned(freq, 4) || !aligned(gq, elem(wb)) || !aligned(gk, elem(wb))) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_cache(const nvfp4_kv_cache* c, const nvfp4_batch* b, int64_t T, const int* status) {
  if (!c || !b) return NVFP4_ERR_NULL;
  if (T < 0 || T > INT32_MAX || c->pages < 0 || c->pages > INT32_MAX || c->heads < 1 || c->heads > 65535 ||
      c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 || c->dim < 32 || c->dim > 256 || c->dim % 32)
    return NVFP4_ERR_SHAPE;
  // any order of page, head and row, each step past what lies below it
  const int64_t counts[3] = {c->pages, c->heads, c->page_size};
  const int64_t strides[2][3] = {{c->code_page, c->code_head, c->code_row}, {c->scale_page, c->scale_head, c->scale_row}};
  for (int k = 0; k < 2; ++k) {
    int o[3] = {0, 1, 2};  // by stride, smallest first; axes of one entry are not stepped over
    for (int i = 0; i < 3; ++i)  // pages and rows are stepped over in the kernels' loops
      if (strides[k][i] < 0 || strides[k][i] > (i == 1 ? kMaxHeadStride : (int64_t)UINT32_MAX)) return NVFP4_ERR_SHAPE;
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (strides[k][o[j]] > strides[k][o[j + 1]]) {
          const int x = o[j];
          o[j] = o[j + 1];
          o[j + 1] = x;
        }
    uint64_t below = k == 0 ? c->dim / 2 : c->dim / 16;  // at most 2^48 + 2^61 + 2^63
    for (int i = 0; i < 3; ++i) {
      const uint64_t n = (uint64_t)counts[o[i]], st = (uint64_t)strides[k][o[i]];
      if (n <= 1) continue;
      if (st < below) return NVFP4_ERR_SHAPE;
      below += (n - 1) * st;
    }
  }
  if (b->sequences < 0 || b->sequences > INT32_MAX - 1 || b->table_width < 0 || b->table_width > INT32_MAX ||
      bad_stride(b->table_stride, b->sequences))
    return NVFP4_ERR_SHAPE;
  if (T > 0 && b->sequences > 0) {
    if (!b->starts || !b->lengths || (b->table_width > 0 && !b->table) || !c->alpha_dev) return NVFP4_ERR_NULL;
    if (c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)) return NVFP4_ERR_NULL;
  }
  for (const uint8_t* p : {c->k_codes, c->v_codes})
    if (!aligned(p, 16)) return NVFP4_ERR_ALIGN;
  for (const uint8_t* p : {c->k_scales, c->v_scales})
    if (!aligned(p, 2)) return NVFP4_ERR_ALIGN;
  if (c->code_page % 16 || c->code_head % 16 || c->code_row % 16 || c->scale_page % 2 || c->scale_head % 2 ||
      c->scale_row % 2)
    return NVFP4_ERR_ALIGN;
  if (!aligned(c->alpha_dev, 4) || !aligned(b->starts, 4) || !aligned(b->lengths, 4) || !aligned(b->table, 4) ||
      !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

nvfp4::CacheView view(const nvfp4_kv_cache* c, const nvfp4_batch* b, int64_t T, int* status) {
  nvfp4::CacheView v;
  v.kc = c->k_codes;
  v.ks = c->k_scales;
  v.vc = c->v_codes;
  v.vs = c->v_scales;
  v.alpha = c->alpha_dev;
  v.ch = c->code_head;
  v.sh = c->scale_head;
  v.cp = (uint32_t)c->code_page;
  v.cr = (uint32_t)c->code_row;
  v.sp = (uint32_t)c->scale_page;
  v.sr = (uint32_t)c->scale_row;
  v.table_width = b->table_width;
  v.table_stride = b->table_stride;
  v.starts = b->starts;
  v.lengths = b->lengths;
  v.table = b->table;
  v.sequences = (int)b->sequences;
  v.pages = (int)c->pages;
  v.heads = c->heads;
  v.page_size = c->page_size;
  v.dim = c->dim;
  v.T = (int)T;
  v.status = status;
  return v;
}

}  // namespace

extern "C" {

int nvfp4_qk_rope(const nvfp4_tokens* q, const nvfp4_tokens* k, int x_is_bf16, int64_t T, int q_heads, int k_heads,
                  int D, int rotated, int interleaved, const int32_t* positions_dev, const float* inv_freq_dev, int norm,
                  float eps, const void* gamma_q_dev, const void* gamma_k_dev, int w_is_bf16, const nvfp4_tokens* out_q,
                  const nvfp4_tokens* out_k, int y_is_bf16, void* stream) {
  const nvfp4_tokens* t[4] = {q, k, out_q, out_k};
  const uintptr_t es[4] = {elem(x_is_bf16), elem(x_is_bf16), elem(y_is_bf16), elem(y_is_bf16)};
  const int st = check_rope(t, es, 4, T, q_heads, k_heads, D, rotated, positions_dev, inv_freq_dev, norm, eps,
                            gamma_q_dev, gamma_k_dev, w_is_bf16);
  if (st) return st;
  if (T == 0 || q_heads + k_heads == 0) return NVFP4_OK;
  nvfp4::RopeArgs a;
  a.q = view(q);
  a.k = view(k);
  a.oq = view(out_q);
  a.ok = view(out_k);
  a.positions = positions_dev;
  a.inv_freq = inv_freq_dev;
  a.gamma_q = gamma_q_dev;
  a.gamma_k = gamma_k_dev;
  a.T = T;
  a.Hq = q_heads;
  a.Hk = k_heads;
  a.D = D;
  a.rotated = rotated;
  a.interleaved = interleaved ? 1 : 0;
  a.norm = norm ? 1 : 0;
  a.in_bf16 = x_is_bf16 ? 1 : 0;
  a.out_bf16 = y_is_bf16 ? 1 : 0;
  a.w_bf16 = w_is_bf16 ? 1 : 0;
  a.eps = eps;
  a.turn = 1.0f;
  return launch_status(nvfp4::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

int64_t nvfp4_qk_rope_backward_workspace(int64_t T, int q_heads, int k_heads, int D) {
  if (bad_rope_sizes(T, q_heads, k_heads, D, 0)) return NVFP4_ERR_SHAPE;
  return T == 0 || q_heads + k_heads == 0 ? 0 : nvfp4::rope_grad_workspace(T, q_heads, k_heads, D);
}

int nvfp4_qk_rope_backward(const nvfp4_tokens* dq, const nvfp4_tokens* dk, int dy_is_bf16, const nvfp4_tokens* q,
                           const nvfp4_tokens* k, int x_is_bf16, int64_t T, int q_heads, int k_heads, int D, int rotated,
                           int interleaved, const int32_t* positions_dev, const float* inv_freq_dev, int norm, float eps,
                           const void* gamma_q_dev, const void* gamma_k_dev, int w_is_bf16, const nvfp4_tokens* dx_q,
                           const nvfp4_tokens* dx_k, float* dgamma_q_dev, float* dgamma_k_dev, void* workspace_dev,
                           int64_t workspace_bytes, void* stream) {
  const nvfp4_tokens* t[6] = {dq, dk, dx_q, dx_k, q, k};
  const uintptr_t xe = elem(x_is_bf16), ye = elem(dy_is_bf16), es[6] = {ye, ye, xe, xe, xe, xe};
  const int st = check_rope(t, es, norm ? 6 : 4, T, q_heads, k_heads, D, rotated, positions_dev, inv_freq_dev, norm, eps,
                            gamma_q_dev, gamma_k_dev, w_is_bf16);
  if (st) return st;
  if (!norm && (dgamma_q_dev || dgamma_k_dev)) return NVFP4_ERR_FLAGS;
  if (!aligned(dgamma_q_dev, 4) || !aligned(dgamma_k_dev, 4)) return NVFP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0 || q_heads + k_heads == 0) {
    const int z = zero(dgamma_q_dev, D * 4, s);
    return z ? z : zero(dgamma_k_dev, D * 4, s);
  }
  nvfp4::RopeGradArgs g;
  nvfp4::RopeArgs& a = g.r;
  a.q = view(dq);
  a.k = view(dk);
  a.oq = view(dx_q);
  a.ok = view(dx_k);
  a.positions = positions_dev;
  a.inv_freq = inv_freq_dev;
  a.gamma_q = gamma_q_dev;
  a.gamma_k = gamma_k_dev;
  a.T = T;
  a.Hq = q_heads;
  a.Hk = k_heads;
  a.D = D;
  a.rotated = rotated;
  a.interleaved = interleaved ? 1 : 0;
  a.norm = norm ? 1 : 0;
  a.in_bf16 = dy_is_bf16 ? 1 : 0;
  a.out_bf16 = x_is_bf16 ? 1 : 0;
  a.w_bf16 = w_is_bf16 ? 1 : 0;
  a.eps = eps;
  a.turn = -1.0f;
  if (!norm) return launch_status(nvfp4::launch_rope(a, s));  // turned back, nothing else
  if (dgamma_q_dev || dgamma_k_dev) {
    const int w = check_workspace(workspace_dev, workspace_bytes, nvfp4::rope_grad_workspace(T, q_heads, k_heads, D));
    if (w) return w;
  }
  g.xq = view(q);
  g.xk = view(k);
  g.dgamma_q = dgamma_q_dev;
  g.dgamma_k = dgamma_k_dev;
  g.ws = static_cast<float*>(workspace_dev);
  return launch_status(nvfp4::launch_rope_grad(g, s));
}

int nvfp4_cache_write(const nvfp4_tokens* k, const nvfp4_tokens* v, int x_is_bf16, int64_t T,
                      const nvfp4_kv_cache* cache, const nvfp4_batch* batch, int* status_dev, void* stream) {
  if (!k || !v) return NVFP4_ERR_NULL;
  const int st = check_cache(cache, batch, T, status_dev);
  if (st) return st;
  if (bad_tokens(k, T, cache->heads) || bad_tokens(v, T, cache->heads)) return NVFP4_ERR_SHAPE;
  const bool empty = T == 0 || batch->sequences == 0;
  if (!empty && (!k->data || !v->data)) return NVFP4_ERR_NULL;
  if (!aligned(k->data, elem(x_is_bf16)) || !aligned(v->data, elem(x_is_bf16))) return NVFP4_ERR_ALIGN;
  if (empty) return NVFP4_OK;
  const nvfp4::CacheCopyArgs a = {view(cache, batch, T, status_dev), view(k), view(v), x_is_bf16 ? 1 : 0};
  return launch_status(nvfp4::launch_cache_write(a, static_cast<cudaStream_t>(stream)));
}

int nvfp4_cache_read(const nvfp4_tokens* k, const nvfp4_tokens* v, int y_is_bf16, int64_t T,
                     const nvfp4_kv_cache* cache, const nvfp4_batch* batch, int* status_dev, void* stream) {
  if (!k || !v) return NVFP4_ERR_NULL;
  const int st = check_cache(cache, batch, T, status_dev);
  if (st) return st;
  if (bad_tokens(k, T, cache->heads) || bad_tokens(v, T, cache->heads)) return NVFP4_ERR_SHAPE;
  if (!aligned(k->data, elem(y_is_bf16)) || !aligned(v->data, elem(y_is_bf16))) return NVFP4_ERR_ALIGN;
  if (T == 0 || batch->sequences == 0 || (!k->data && !v->data)) return NVFP4_OK;
  const nvfp4::CacheCopyArgs a = {view(cache, batch, T, status_dev), view(k), view(v), y_is_bf16 ? 1 : 0};
  return launch_status(nvfp4::launch_cache_read(a, static_cast<cudaStream_t>(stream)));
}

int64_t nvfp4_cache_attention_workspace(int64_t T, int q_heads, int heads, int dim, int64_t sequences) {
  if (T < 0 || T > INT32_MAX || heads < 1 || heads > 65535 || q_heads < 1 || q_heads > 65535 || q_heads % heads ||
      dim < 32 || dim > 256 || dim % 32 || sequences < 0 || sequences > INT32_MAX - 1)
    return NVFP4_ERR_SHAPE;
  return T == 0 || sequences == 0 ? 0 : nvfp4::attend_workspace(T, q_heads, heads, dim, sequences);
}

int nvfp4_cache_attention(const nvfp4_tokens* q, int64_t T, int q_heads, const nvfp4_kv_cache* cache,
                          const nvfp4_batch* batch, float scale, int causal, int64_t window, int64_t sinks,
                          const nvfp4_tokens* o, float* lse_dev, void* workspace_dev, int64_t workspace_bytes,
                          int* status_dev, void* stream) {
  if (!q || !o) return NVFP4_ERR_NULL;
  const int st = check_cache(cache, batch, T, status_dev);
  if (st) return st;
  if (q_heads < 1 || q_heads > 65535 || q_heads % cache->heads || bad_tokens(q, T, q_heads) || bad_tokens(o, T, q_heads))
    return NVFP4_ERR_SHAPE;
  if (std::isnan(scale) || std::isinf(scale) || window < 0 || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX ||
      (!causal && window > 0) || (window == 0 && sinks > 0))
    return NVFP4_ERR_FLAGS;
  const bool empty = T == 0 || batch->sequences == 0;
  if (!empty && (!q->data || !o->data)) return NVFP4_ERR_NULL;
  if (!aligned(q->data, 2) || !aligned(o->data, 2) || !aligned(lse_dev, 4)) return NVFP4_ERR_ALIGN;
  if (empty) return NVFP4_OK;
  const int w = check_workspace(workspace_dev, workspace_bytes,
                                nvfp4::attend_workspace(T, q_heads, cache->heads, cache->dim, batch->sequences));
  if (w) return w;
  nvfp4::AttendArgs a;
  a.c = view(cache, batch, T, status_dev);
  a.q = view(q);
  a.o = view(o);
  a.lse = lse_dev;
  a.ws = static_cast<float*>(workspace_dev);
  a.Hq = q_heads;
  a.group = q_heads / cache->heads;
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  a.window = (int)window;
  a.sinks = (int)sinks;
  a.few_rows = nvfp4::attend_few_rows(T, a.group, cache->heads, batch->sequences);
  return launch_status(nvfp4::launch_attend(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
