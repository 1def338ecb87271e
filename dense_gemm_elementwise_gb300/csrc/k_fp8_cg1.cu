#include "fp8_kernel.cuh"
namespace ge {
const void *fp8_kernel_cg1(bool square, bool add, bool turned) {
  return square ? pick_fp8<1, 128, true>(add, turned) : pick_fp8<1, 128, false>(add, turned);
}
}  // namespace ge
