// nvfp4_attention_selftest.cu -- test-only entry of the attention kernel for many rows in a
// build whose filling warps report four blocks of keys and no more (NVFP4_TEST_NO_COPIES): its waits run out.
#include <cuda_runtime.h>

#include "attend.cuh"

extern "C" __attribute__((visibility("default"))) int nvfp4_selftest_attend_many(
    void* q, void* o, uint8_t* kc, uint8_t* ks, uint8_t* vc, uint8_t* vs, const float* alpha, const int* starts,
    const int* lengths, const int* table, int T, int heads, int group, int dim, int page_size, int pages, int* status) {
  nvfp4::AttendArgs a = {};
  nvfp4::CacheView& c = a.c;
  c.kc = kc;
  c.ks = ks;
  c.vc = vc;
  c.vs = vs;
  c.alpha = alpha;
  c.cr = (uint32_t)dim / 2;
  c.ch = (int64_t)page_size * c.cr;
  c.cp = (uint32_t)(heads * c.ch);
  c.sr = (uint32_t)dim / 16;
  c.sh = (int64_t)page_size * c.sr;
  c.sp = (uint32_t)(heads * c.sh);
  c.table_width = c.table_stride = pages;
  c.starts = starts;
  c.lengths = lengths;
  c.table = table;
  c.sequences = 1;
  c.pages = pages;
  c.heads = heads;
  c.page_size = page_size;
  c.dim = dim;
  c.T = T;
  c.status = status;
  a.Hq = heads * group;
  a.group = group;
  a.q = {q, (int64_t)a.Hq * dim, dim};
  a.o = {o, (int64_t)a.Hq * dim, dim};
  a.scale = 0.1f;
  a.causal = 1;
  return (int)nvfp4::launch_attend_many(a, nullptr);
}
