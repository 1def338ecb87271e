#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_whole_pairs(int dt, int nv, int threads) {
  if (nv == 1) return threads <= kVecThreads ? pick_grad<1, P_PAIRS, kVecThreads, true>(dt) : pick_grad<1, P_PAIRS, kMaxThreads, true>(dt);
  return pick_grad<2, P_PAIRS, kMaxThreads, true>(dt);
}
}  // namespace ge
