// as with e4m3
#define GE_MOE_GROUPS 2
#include "moe_kernel.cuh"
namespace ge {
MoeKernel moe_experts_e5m2(int xt) {
  return {xt == GE_BF16 ? reinterpret_cast<const void *>(moe_experts_kernel<GE_BF16, GE_E5M2>)
                        : reinterpret_cast<const void *>(moe_experts_kernel<GE_F16, GE_E5M2>),
          kThreads, kMoeSmem};
}
}  // namespace ge
