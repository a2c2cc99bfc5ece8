// attention_internal.h -- kernel launch interface of the attention operators, shared by
// libnvfp4_attention's translation units.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "nvfp4_attention.h"

namespace nvfp4 {

// A token tensor: element (t, h, d) at p[t * ts + h * hs + d].
struct Tokens {
  void* p;
  int64_t ts, hs;
};

struct RopeArgs {
  Tokens q, k;    // what is turned: the inputs, or the gradients of the outputs
  Tokens oq, ok;  // outputs
  const int32_t* positions;
  const float* inv_freq;
  const void* gamma_q;  // nullable
  const void* gamma_k;  // nullable
  int64_t T;
  int Hq, Hk, D, rotated;
  int interleaved, norm, in_bf16, out_bf16, w_bf16;
  float eps;
  float turn;  // 1, or -1 to turn back
};

struct RopeGradArgs {
  RopeArgs r;     // q, k: the gradients of the outputs; oq, ok: those of the inputs (out_bf16 is also x's type)
  Tokens xq, xk;  // the forward pass's inputs
  float* dgamma_q;  // nullable
  float* dgamma_k;  // nullable
  float* ws;
};

// The batch and the cache as kernels take them.
struct CacheView {
  uint8_t *kc, *ks, *vc, *vs;
  const float* alpha;
  int64_t ch, sh;           // strides of codes and scales in bytes: head,
  uint32_t cp, cr, sp, sr;  // page and row
  int64_t table_width, table_stride;
  const int32_t *starts, *lengths, *table;
  int sequences, pages, heads, page_size, dim;
  int T;
  int* status;  // nullable
};

struct CacheCopyArgs {
  CacheView c;
  Tokens k, v;  // a null p: not wanted (read only)
  int bf16;
};

struct AttendArgs {
  CacheView c;
  Tokens q, o;
  float* lse;  // nullable
  float* ws;
  int Hq, group;  // query heads, and of those how many read one key head
  float scale;
  int causal;
  int window, sinks;
  int few_rows;  // the most rows of a sequence that the kernel for few takes
};

int64_t rope_grad_workspace(int64_t T, int Hq, int Hk, int D);
int attend_few_rows(int64_t T, int group, int heads, int64_t sequences);
int64_t attend_workspace(int64_t T, int Hq, int heads, int dim, int64_t sequences);

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_grad(const RopeGradArgs& a, cudaStream_t s);
cudaError_t launch_cache_write(const CacheCopyArgs& a, cudaStream_t s);
cudaError_t launch_cache_read(const CacheCopyArgs& a, cudaStream_t s);
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s);

}  // namespace nvfp4
