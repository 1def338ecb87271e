// xent_math.cuh -- 2^x and roundings of the vocabulary loss's kernels.
#pragma once

#include <stdint.h>

namespace ge {

// 2^x to 2^-22, subnormal results as 0
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two values rounded to 16 bits, lo in the lower half
__device__ __forceinline__ uint32_t pack16(bool bf16, float lo, float hi) {
  uint32_t r;
  if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace ge
