#include "fp8_kernel.cuh"
namespace ge { const void *fp8_kernel_cg2(bool square) { return pick_fp8<2, 256>(square); } }
