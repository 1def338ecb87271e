#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_run_odd(int dt, int nv, int threads) {
  if (dt == GE_F16) {
    if (nv == 1) return threads <= kVecThreads ? run_of<GE_F16, 1, P_STRIDED, kVecThreads>() : run_of<GE_F16, 1, P_STRIDED, kMaxThreads>();
    return run_of<GE_F16, 2, P_STRIDED, kMaxThreads>();
  }
  if (nv == 1) return threads <= kVecThreads ? run_of<GE_BF16, 1, P_STRIDED, kVecThreads>() : run_of<GE_BF16, 1, P_STRIDED, kMaxThreads>();
  return run_of<GE_BF16, 2, P_STRIDED, kMaxThreads>();
}
}  // namespace ge
