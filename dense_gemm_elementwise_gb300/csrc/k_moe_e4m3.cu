// two groups: conversions need more warps to fill their waits (64 tokens, 128 experts of 4096 x 2048 in 725 us
// against 791 with one)
#define GE_MOE_GROUPS 2
#include "moe_kernel.cuh"
namespace ge {
MoeKernel moe_experts_e4m3(int xt) {
  return {xt == GE_BF16 ? reinterpret_cast<const void *>(moe_experts_kernel<GE_BF16, GE_E4M3>)
                        : reinterpret_cast<const void *>(moe_experts_kernel<GE_F16, GE_E4M3>),
          kThreads, kMoeSmem};
}
}  // namespace ge
