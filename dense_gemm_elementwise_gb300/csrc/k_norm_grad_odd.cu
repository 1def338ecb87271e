#include "norm_kernel.cuh"
namespace ge {
const void *norm_kernel_grad_odd(int dt, int nv, int threads) {
  if (dt == GE_F16) {
    if (nv == 1) return threads <= kVecThreads ? grad_of<GE_F16, 1, P_STRIDED, kVecThreads, false>() : grad_of<GE_F16, 1, P_STRIDED, kMaxThreads, false>();
    return grad_of<GE_F16, 2, P_STRIDED, kMaxThreads, false>();
  }
  if (nv == 1) return threads <= kVecThreads ? grad_of<GE_BF16, 1, P_STRIDED, kVecThreads, false>() : grad_of<GE_BF16, 1, P_STRIDED, kMaxThreads, false>();
  return grad_of<GE_BF16, 2, P_STRIDED, kMaxThreads, false>();
}
}  // namespace ge
