// one group: with two, 8 tokens and 32 experts of 4096 x 1536 take 151 us instead of 143
#define GE_MOE_GROUPS 1
#include "moe_kernel.cuh"
namespace ge {
MoeKernel moe_experts_16(int xt) {
  return {xt == GE_BF16 ? reinterpret_cast<const void *>(moe_experts_kernel<GE_BF16, GE_BF16>)
                        : reinterpret_cast<const void *>(moe_experts_kernel<GE_F16, GE_F16>),
          kThreads, kMoeSmem};
}
}  // namespace ge
