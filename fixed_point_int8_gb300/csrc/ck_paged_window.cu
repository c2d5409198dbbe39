// Attention of a few new tokens over a window of the cache.
#include "ck_paged_few.cuh"

namespace ck {

cudaError_t launch_few_window(const FewParams& p, const FewPlan& w, const DeviceFacts& f, cudaStream_t s) {
  return launch_few_any<true>(p, w, f, s);
}

}  // namespace ck
