#include "fp8_kernel.cuh"
namespace ge { const void *fp8_kernel_cg1(bool square) { return pick_fp8<1, 128>(square); } }
