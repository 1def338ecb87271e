#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_run(int dt, int nv, bool vec) {
  if (nv == 1) return vec ? pick_run<1, true>(dt) : pick_run<1, false>(dt);
  return vec ? pick_run<2, true>(dt) : pick_run<2, false>(dt);
}
}  // namespace ge
