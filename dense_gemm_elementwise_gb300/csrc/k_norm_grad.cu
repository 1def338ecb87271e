#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad(int dt, int nv, bool vec) {
  if (nv == 1) return vec ? pick_grad<1, true, false>(dt) : pick_grad<1, false, false>(dt);
  return vec ? pick_grad<2, true, false>(dt) : pick_grad<2, false, false>(dt);
}
}  // namespace ge
