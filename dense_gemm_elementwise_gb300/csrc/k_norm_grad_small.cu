#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_small(int dt, int nv, int threads, bool even) {
  const bool wide = threads > kVecThreads;
  if (even) {
    if (nv == 1) return pick_grad<1, P_PAIRS, kVecThreads, false>(dt);
    return wide ? pick_grad<2, P_PAIRS, kMaxThreads, false>(dt) : pick_grad<2, P_PAIRS, kVecThreads, false>(dt);
  }
  if (nv == 1) return grad_of<GE_F32, 1, P_STRIDED, kVecThreads, false>();
  return wide ? grad_of<GE_F32, 2, P_STRIDED, kMaxThreads, false>() : grad_of<GE_F32, 2, P_STRIDED, kVecThreads, false>();
}
}  // namespace ge
