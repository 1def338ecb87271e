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

// a launch with programmatic stream serialization
inline cudaError_t launch_pdl(const void *fn, dim3 grid, dim3 block, int smem, void **args, cudaStream_t s,
                              int cluster = 1) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

inline bool is_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

}  // namespace ge
