#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_whole(int dt, int nv, bool vec) {
  if (nv == 1) return vec ? pick_grad<1, true, true>(dt) : pick_grad<1, false, true>(dt);
  return vec ? pick_grad<2, true, true>(dt) : pick_grad<2, false, true>(dt);
}
}  // namespace ge
