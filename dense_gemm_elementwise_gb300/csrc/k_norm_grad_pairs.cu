#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_pairs(int dt, int nv, int threads) {
  if (nv == 1) return threads <= kVecThreads ? pick_grad<1, P_PAIRS, kVecThreads, false>(dt) : pick_grad<1, P_PAIRS, kMaxThreads, false>(dt);
  return pick_grad<2, P_PAIRS, kMaxThreads, false>(dt);
}
}  // namespace ge
