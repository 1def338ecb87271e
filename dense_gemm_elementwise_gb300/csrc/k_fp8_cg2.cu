#include "fp8_kernel.cuh"
namespace ge {
const void *fp8_kernel_cg2(bool square, bool turned) {
  return square ? pick_fp8<2, 256, true>(turned) : pick_fp8<2, 256, false>(turned);
}
}  // namespace ge
