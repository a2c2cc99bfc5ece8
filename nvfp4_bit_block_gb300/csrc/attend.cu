// attend.cu -- attention of a batch's queries to the NVFP4 cache.
//
// For each row (token and query head), with the running maximum m and sum l of a softmax
// over the visible keys j: o = sum exp(s_j - m) v_j / l, lse = m + log l.  Sequences with few
// rows to a key head are bound by the cache's bytes (attend_few.cu), those with many by their
// products (attend_many.cu).  The lengths are on the device: where a batch may hold both, both
// kernels run, and each leaves the other's sequences alone.
#include "attend.cuh"

namespace nvfp4 {

int64_t attend_workspace(int64_t T, int Hq, int heads, int dim, int64_t sequences) {
  return attend_few_workspace(T, Hq / heads, dim, sequences);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_attend_few(a, s);
  if (e != cudaSuccess || a.c.T <= 1 || (int64_t)a.c.T * a.group <= attention::kFewRows) return e;
  return launch_attend_many(a, s);
}

}  // namespace nvfp4
