#include "fp8_kernel.cuh"
namespace ge {
const void *fp8_kernel_cg2(bool square, bool add, bool turned) {
  return square ? pick_fp8<2, 256, true>(add, turned) : pick_fp8<2, 256, false>(add, turned);
}
}  // namespace ge
