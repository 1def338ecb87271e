#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_whole(int dt, int nv) {
  return nv == 1 ? pick_grad<1, P_RING, kVecThreads, true>(dt) : nv == 2 ? pick_grad<2, P_RING, kVecThreads, true>(dt) : pick_grad<4, P_DIRECT, kVecThreads, true>(dt);
}
}  // namespace ge
