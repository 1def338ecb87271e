#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_run(int dt, int nv) {
  return nv == 1 ? pick_run<1, P_RING, kRunBound>(dt) : nv == 2 ? pick_run<2, P_RING, kRunBound>(dt) : pick_run<4, P_DIRECT, kVecThreads>(dt);
}
}  // namespace ge
