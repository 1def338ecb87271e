// moe.cu -- host side of the expert layer for a few tokens (gemm_epi_moe_*), its router's kernel and its choice's; the
// experts' is in moe_kernel.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "gemm_epi.h"
#include "host.h"
#include "moe.h"
#include "moe_choice.cuh"
#include "ptx.cuh"

using namespace ge;

namespace {

constexpr int kRouterTokens = 4, kRouterWarps = 16;  // warps at most: 8 columns a thread, up to 4096 columns at once

// a + b as a sum and what its rounding left (exact)
__device__ __forceinline__ void two_sum(float &s, float &e, float x) {
  const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
  s = t;
}

template <int XT>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (XT == GE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// A CTA: one expert and four tokens; its warps share the columns.
template <int XT, bool F32>
__global__ void __launch_bounds__(32 * kRouterWarps) moe_router_kernel(const __grid_constant__ MoeParams p) {
  __shared__ float2 part[kRouterWarps][kRouterTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    p.done[e] = 0;
    if (e == 0) *p.head = MoeHead{0, 0};
  }
  if (blockIdx.y == 0)
    for (int i = e * blockDim.x + threadIdx.x; i < (p.D + kDownCols - 1) / kDownCols; i += p.E * blockDim.x) p.shares[i] = 0;
  float s[kRouterTokens] = {}, r[kRouterTokens] = {};
  const uint16_t *x = static_cast<const uint16_t *>(p.x);
  for (int d = 8 * threadIdx.x; d < p.D; d += 8 * blockDim.x) {
    float w[8];
    if constexpr (F32) {
      const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p.w_router) + int64_t(e) * p.D + d);
      const float4 a = __ldg(q), b = __ldg(q + 1);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.w_router) + int64_t(e) * p.D + d));
      const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack<XT>(q[j]);
        w[2 * j] = f.x;
        w[2 * j + 1] = f.y;
      }
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
      if (t0 + t >= p.T) break;
      const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x + int64_t(t0 + t) * p.ldx + d));
      const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack<XT>(q[j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a0 = h ? f.y : f.x, b0 = w[2 * j + h];
          // products of two 16-bit values are exact
          const float m = __fmul_rn(a0, b0);
          two_sum(s[t], r[t], m);
          if constexpr (F32) r[t] = __fadd_rn(r[t], __fmaf_rn(a0, b0, -m));
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kRouterTokens; ++t) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float so = __shfl_xor_sync(0xffffffffu, s[t], o), ro = __shfl_xor_sync(0xffffffffu, r[t], o);
      two_sum(s[t], r[t], so);
      r[t] = __fadd_rn(r[t], ro);
    }
    if (lane == 0) part[warp][t] = make_float2(s[t], r[t]);
  }
  __syncthreads();
  if (threadIdx.x < kRouterTokens && t0 + threadIdx.x < p.T) {
    float2 a = part[0][threadIdx.x];
#pragma unroll 4
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) {
      const float2 b = part[w][threadIdx.x];
      two_sum(a.x, a.y, b.x);
      a.y = __fadd_rn(a.y, b.y);
    }
    const float hi = __fadd_rn(a.x, a.y);
    // (infinities and NaN have no remainder)
    const float lo = isfinite(hi) ? __fsub_rn(a.y, __fsub_rn(hi, a.x)) : 0.f;
    p.logits[int64_t(t0 + threadIdx.x) * p.E + e] = make_float2(isfinite(a.x) ? hi : a.x, lo);
  }
}

// A warp: one token's experts.
__global__ void __launch_bounds__(32) moe_choice_kernel(const __grid_constant__ MoeParams p) {
  __shared__ ChoiceSpace space;
  griddep_wait();
  griddep_launch_dependents();
  choose(p, blockIdx.x, p.expert, p.share, space, true);
}

}  // namespace

struct gemm_epi_moe_plan {
  MoeParams p;
  const void *router;
  MoeKernel experts;
  int grid;
  bool k8;
  bool apart;  // the choice has a launch of its own
};

namespace {

struct Space {
  size_t done, shares, logits, expert, share, h, part, bytes;
};

Space space_of(const MoeParams &p) {
  Space s;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t pairs = static_cast<size_t>(p.T) * static_cast<size_t>(p.k);
  s.done = take(sizeof(uint32_t) * static_cast<size_t>(p.E));
  s.shares = take(sizeof(uint32_t) * static_cast<size_t>(ceil_div(p.D, kDownCols)));
  s.logits = take(sizeof(float2) * static_cast<size_t>(p.T) * static_cast<size_t>(p.E));
  s.expert = take(sizeof(uint16_t) * pairs);
  s.share = take(sizeof(float) * pairs);
  s.h = take(2 * sizeof(uint16_t) * pairs * static_cast<size_t>(p.F));
  s.part = take(sizeof(float) * pairs * static_cast<size_t>(p.D));
  s.bytes = at;
  return s;
}

}  // namespace

extern "C" {

int gemm_epi_moe_plan_create(gemm_epi_moe_plan **plan, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k,
                             const ge_moe_desc *desc) {
  if (!plan) return GE_ERR_INVALID;
  *plan = nullptr;
  if (!desc) return GE_ERR_INVALID;
  const ge_moe_desc &d = *desc;
  const bool k8 = d.w == GE_E4M3 || d.w == GE_E5M2;
  if ((d.x != GE_F16 && d.x != GE_BF16) || (d.w != d.x && !k8) || (d.router != d.x && d.router != GE_F32))
    return GE_ERR_UNSUPPORTED;
  if (d.act != 0 && d.act != GE_SILU && d.act != GE_GELU && d.act != GE_RELU) return GE_ERR_UNSUPPORTED;
  if ((d.score != GE_SCORE_SOFTMAX && d.score != GE_SCORE_SIGMOID) || (d.renormalise != 0 && d.renormalise != 1) ||
      d.timeout_ms < 0 || (d.debug_flags & ~GE_DEBUG_SKIP_FIRST_LOAD) != 0 || !std::isfinite(d.route_scale) ||
      d.reserved != 0)
    return GE_ERR_INVALID;
  if (T <= 0 || T > GE_MOE_MAX_TOKENS || E <= 0 || E > GE_MOE_MAX_EXPERTS || k <= 0 || k > E || k > GE_MOE_MAX_K ||
      D <= 0 || D > (1 << 20) || F <= 0 || F > (1 << 20))
    return GE_ERR_SHAPE;
  const int64_t ldx = d.ldx ? d.ldx : D, ldy = d.ldy ? d.ldy : D;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  if (ldx < D || ldy < D || ldx > kMost || ldy > kMost) return GE_ERR_SHAPE;
  const int64_t unit = k8 ? 16 : 8;
  if (D % unit != 0 || F % unit != 0 || ldx % 8 != 0 || ldy % 8 != 0) return GE_ERR_MISALIGNED;
  int dev = 0, sms = 0, smem = 0;
  const int st = current_device(&dev, &sms, &smem);
  if (st != GE_OK) return st;
  gemm_epi_moe_plan *pl = new (std::nothrow) gemm_epi_moe_plan();
  if (!pl) return GE_ERR_INVALID;
  MoeParams &p = pl->p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  p.T = static_cast<int32_t>(T);
  p.D = static_cast<int32_t>(D);
  p.F = static_cast<int32_t>(F);
  p.E = static_cast<int32_t>(E);
  p.k = static_cast<int32_t>(k);
  p.ldx = ldx;
  p.ldy = ldy;
  p.score = d.score;
  p.renormalise = d.renormalise;
  p.act = d.act ? d.act : GE_SILU;
  p.route_scale = d.route_scale == 0.f ? 1.f : d.route_scale;
  p.debug_flags = d.debug_flags;
  p.timeout_ns = uint64_t(d.timeout_ms > 0 ? d.timeout_ms : 1000) * 1000000u;
  p.status = status_block();
  pl->k8 = k8;
  pl->experts = d.w == GE_E4M3 ? moe_experts_e4m3(d.x) : d.w == GE_E5M2 ? moe_experts_e5m2(d.x) : moe_experts_16(d.x);
  const bool f32 = d.router == GE_F32;
  if (d.x == GE_BF16)
    pl->router = f32 ? reinterpret_cast<const void *>(moe_router_kernel<GE_BF16, true>)
                     : reinterpret_cast<const void *>(moe_router_kernel<GE_BF16, false>);
  else
    pl->router = f32 ? reinterpret_cast<const void *>(moe_router_kernel<GE_F16, true>)
                     : reinterpret_cast<const void *>(moe_router_kernel<GE_F16, false>);
  // The choice is a launch of its own where a CTA of the experts' kernel has fewer warps than there are tokens (64 tokens and 128
  // experts of 4096 x 2048 in 8 bits 743 -> 723 us, 29 and 13 of 1000 x 520 32.4 -> 30.2; one token and 64 of 2048 x 1024 27.1 against 28.3).
  pl->apart = T > pl->experts.threads / 32;
  int per_sm = 0;
  if (!p.status ||
      cudaFuncSetAttribute(pl->experts.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, pl->experts.smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, pl->experts.fn, pl->experts.threads,
                                                    static_cast<size_t>(pl->experts.smem)) != cudaSuccess ||
      per_sm < 1) {
    cudaGetLastError();
    delete pl;
    return GE_ERR_CUDA;
  }
  const int64_t most = std::min<int64_t>(E, T * k) * (ceil_div(F, kUpCols) + ceil_div(D, kDownCols));
  pl->grid = static_cast<int>(std::min<int64_t>(int64_t(per_sm) * sms, most));
  *plan = pl;
  return GE_OK;
}

void gemm_epi_moe_plan_destroy(gemm_epi_moe_plan *plan) { delete plan; }

size_t gemm_epi_moe_workspace_bytes(const gemm_epi_moe_plan *plan) { return plan ? space_of(plan->p).bytes : 0; }

int gemm_epi_moe_run(gemm_epi_moe_plan *pl, const void *x, const void *w_router, const float *bias, const void *w_gate_up,
                     const float *s_gate_up, const void *w_down, const float *s_down, void *y, int32_t *index, float *weight,
                     void *workspace, size_t workspace_bytes, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  if (!x || !w_router || !w_gate_up || !w_down || !y || (pl->k8 && (!s_gate_up || !s_down))) return GE_ERR_MISSING_ARG;
  if (!pl->k8 && (s_gate_up || s_down)) return GE_ERR_INVALID;
  for (const void *q : {x, w_router, static_cast<const void *>(bias), w_gate_up, static_cast<const void *>(s_gate_up), w_down,
                        static_cast<const void *>(s_down), static_cast<const void *>(y), static_cast<const void *>(index),
                        static_cast<const void *>(weight)})
    if (!is_aligned16(q)) return GE_ERR_MISALIGNED;
  const Space s = space_of(pl->p);
  if (!workspace || workspace_bytes < s.bytes) return GE_ERR_WORKSPACE;
  if (!is_aligned16(workspace)) return GE_ERR_MISALIGNED;
  MoeParams p = pl->p;
  p.x = x;
  p.w_router = w_router;
  p.bias = bias;
  p.w_up = w_gate_up;
  p.s_up = s_gate_up;
  p.w_down = w_down;
  p.s_down = s_down;
  p.y = y;
  p.index = index;
  p.weight = weight;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.head = reinterpret_cast<MoeHead *>(ws);
  p.done = reinterpret_cast<uint32_t *>(ws + s.done);
  p.shares = reinterpret_cast<uint32_t *>(ws + s.shares);
  p.logits = reinterpret_cast<float2 *>(ws + s.logits);
  p.expert = pl->apart ? reinterpret_cast<uint16_t *>(ws + s.expert) : nullptr;
  p.share = reinterpret_cast<float *>(ws + s.share);
  p.h = reinterpret_cast<uint16_t *>(ws + s.h);
  p.part = reinterpret_cast<float *>(ws + s.part);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *args[] = {&p};
  if (launch_pdl(pl->router, dim3(static_cast<unsigned>(p.E), static_cast<unsigned>(ceil_div(p.T, kRouterTokens))),
                 dim3(static_cast<unsigned>(std::min<int64_t>(32 * kRouterWarps, round_up(ceil_div(p.D, 8), 32)))), 0, args, st) != cudaSuccess)
    return GE_ERR_CUDA;
  if (pl->apart &&
      launch_pdl(reinterpret_cast<const void *>(moe_choice_kernel), dim3(static_cast<unsigned>(p.T)), dim3(32), 0, args, st) != cudaSuccess)
    return GE_ERR_CUDA;
  return launch_pdl(pl->experts.fn, dim3(static_cast<unsigned>(pl->grid)), dim3(pl->experts.threads), pl->experts.smem, args, st) == cudaSuccess
             ? GE_OK
             : GE_ERR_CUDA;
}

}  // extern "C"
