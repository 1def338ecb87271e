#include "xent_kernel.cuh"
namespace ge { const void *xent_kernel_cg2(int mode) { return pick_xent<2, 256>(mode); } }
