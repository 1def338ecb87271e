#include "xent_kernel.cuh"
namespace ge { const void *xent_kernel_cg1(int mode) { return pick_xent<1, 128>(mode); } }
