#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_run(int dt, int nv, int threads, bool vec) {
  if (vec) return nv == 1 ? pick_run<1, P_RING, kRunBound>(dt) : nv == 2 ? pick_run<2, P_RING, kRunBound>(dt) : pick_run<4, P_DIRECT, kVecThreads>(dt);
  if (nv == 1) return threads <= kVecThreads ? pick_run<1, P_STRIDED, kVecThreads>(dt) : pick_run<1, P_STRIDED, kMaxThreads>(dt);
  return pick_run<2, P_STRIDED, kMaxThreads>(dt);
}
}  // namespace ge
