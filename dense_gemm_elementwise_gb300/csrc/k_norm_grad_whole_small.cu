#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_whole_small(int dt, int nv, int threads, bool even) {
  const bool wide = threads > kVecThreads;
  if (even) {
    if (nv == 1) return pick_grad<1, P_PAIRS, kVecThreads, true>(dt);
    return wide ? pick_grad<2, P_PAIRS, kMaxThreads, true>(dt) : pick_grad<2, P_PAIRS, kVecThreads, true>(dt);
  }
  if (nv == 1) return grad_of<GE_F32, 1, P_STRIDED, kVecThreads, true>();
  return wide ? grad_of<GE_F32, 2, P_STRIDED, kMaxThreads, true>() : grad_of<GE_F32, 2, P_STRIDED, kVecThreads, true>();
}
}  // namespace ge
