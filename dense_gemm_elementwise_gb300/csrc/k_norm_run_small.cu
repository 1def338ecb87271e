#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_run_small(int dt, int nv, int threads, bool even) {
  const bool wide = threads > kVecThreads;
  if (even) {
    if (nv == 1) return pick_run<1, P_PAIRS, kRunBound>(dt);
    return wide ? pick_run<2, P_PAIRS, kMaxThreads>(dt) : pick_run<2, P_PAIRS, kRunBound>(dt);
  }
  if (nv == 1) return run_of<GE_F32, 1, P_STRIDED, kRunBound>();
  return wide ? run_of<GE_F32, 2, P_STRIDED, kMaxThreads>() : run_of<GE_F32, 2, P_STRIDED, kRunBound>();
}
}  // namespace ge
