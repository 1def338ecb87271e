// moe.h -- parameters and handles of the experts' kernel.
#pragma once

#include <cuda_runtime_api.h>

#include <stdint.h>

#include "gemm_epi.h"

namespace ge {

constexpr int kPairs = GE_MOE_MAX_TOKENS * GE_MOE_MAX_K;
constexpr int kUpCols = 16, kDownCols = 32;  // a unit's columns of h, of y

struct MoeHead {
  uint32_t ticket, abort;
};

struct MoeParams {
  const void *x, *w_router;
  const float *bias;
  const void *w_up;
  const float *s_up;
  const void *w_down;
  const float *s_down;
  void *y;
  int32_t *index;
  float *weight;
  MoeHead *head;
  uint32_t *done;   // units of the first kind, by expert
  uint32_t *shares;  // experts that have added their share of kDownCols columns of y
  float2 *logits;   // (T, E)
  uint16_t *expert;  // the choice (T, k), where it has a kernel of its own, and
  float *share;      // ... its weights
  uint16_t *h;      // (T k, F) twice: values, and what their rounding left
  float *part;      // (T k, D)
  uint32_t *status;
  uint64_t timeout_ns;
  int64_t ldx, ldy;
  int32_t T, D, F, E, k;
  int32_t score, renormalise, act;
  float route_scale;
  uint32_t debug_flags;
};

struct MoeKernel {
  const void *fn;
  int threads, smem;
};

// x's type, and the weights': the same, GE_E4M3 or GE_E5M2
MoeKernel moe_experts_16(int xt);
MoeKernel moe_experts_e4m3(int xt);
MoeKernel moe_experts_e5m2(int xt);

}  // namespace ge
