// host.h -- host helpers of plan.cu that the operators beside the GEMM share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <stdint.h>

namespace ge {

// current device: index, SM count, shared memory one CTA may ask for.
// GE_ERR_ARCH unless it has compute capability 10.3.
int current_device(int *dev, int *sms, int *max_smem);

// the device status block (timeouts) of the current device, nullptr on failure
uint32_t *status_block();

// 2-D tensor (d0 contiguous, d1 rows `pitch` elements apart, d2 slices `slice` elements
// apart) with a (b0, b1, 1) box of 128-byte rows, 128-byte swizzle
bool encode_rows(CUtensorMap *m, int dtype, const void *ptr, uint64_t d0, uint64_t d1, uint64_t d2,
                 uint64_t pitch, uint64_t slice, uint32_t b0, uint32_t b1);

inline bool is_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

}  // namespace ge
