#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_run_pairs(int dt, int nv, int threads) {
  if (nv == 1) return threads <= kVecThreads ? pick_run<1, P_PAIRS, kVecThreads>(dt) : pick_run<1, P_PAIRS, kMaxThreads>(dt);
  return pick_run<2, P_PAIRS, kMaxThreads>(dt);
}
}  // namespace ge
