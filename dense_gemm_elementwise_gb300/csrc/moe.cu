// moe.cu -- a mixture-of-experts layer for a few tokens (gemm_epi_moe_*), in two launches.
//
//   router   l = x w_router^T, in pairs of fp32 (TwoSum): the choice of experts has to be that
//            of exact logits, or a token's output is another's
//   experts  every CTA chooses the experts from the logits (cheaper than a third launch or
//            a grid-wide wait), then takes units of work by ticket:
//              1. 8 columns of h = act(gate) * up of one expert: 8 gate and 8 up rows against
//                 the tokens that chose it
//              2. 16 columns of y's share of one expert: 16 rows of w_down against its h,
//                 times the routing weight; the last unit of those 16 columns adds the
//                 experts' shares in the order of the choice
//            A unit of the second kind waits for its expert's units of the first kind.
//            Tickets rise, so those are all held by CTAs that run and wait for nothing:
//            no CTA has to be resident for another to finish.
//
// Few tokens leave the tensor unit idle: the layer is bound by reading the chosen experts'
// weights once.  So a CTA's warps are there to keep that reading going:
//   producer  takes tickets and copies their rows, 2 KiB of 16 rows at a time, into a ring of
//             shared memory (bulk copies), several units ahead of
//   eight consumers, which share a stage's columns and multiply them by mma.sync (tcgen05 would want
//             128 rows of tokens): a lane reads 16 consecutive bytes of a row, and what it holds
//             is called columns 2q, 2q + 1, 2q + 8, 2q + 9 of a step; the tokens' side is read
//             the same way, so the sum runs over the same columns
//   watcher   waits for the h of units that are still on their way into the ring
//   finisher  tells the GPU that a unit is done, and adds the shares of y
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "gemm_epi.h"
#include "host.h"
#include "ptx.cuh"
#include "xent_math.cuh"

using namespace ge;

namespace {

constexpr int kPairs = GE_MOE_MAX_TOKENS * GE_MOE_MAX_K;
constexpr int kWarps = 8;           // consumers; then the producer, the watcher and the finisher
constexpr int kProducer = kWarps, kWatcher = kWarps + 1, kFinisher = kWarps + 2;
constexpr int kThreads = 32 * (kWarps + 3);
constexpr int kBlock = 128;        // columns that share a scale
constexpr int kTile = 8;           // tokens of one mma
constexpr int kRoundTiles = 2;     // of them whose sums are joined at a time
constexpr int kSegment = 2048;     // bytes of a row in a stage
constexpr int kPitch = kSegment + 64;  // lanes of two rows touch different banks
constexpr int kStages = 5;
constexpr int kQueue = 8;          // units under way in a CTA
constexpr int kUpCols = 8, kDownCols = 16;  // a unit's columns of h, of y
constexpr int kRouterTokens = 4, kRouterWarps = 4;

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
  uint32_t *shares;  // experts' shares of 16 columns of y
  float2 *logits;   // (T, E)
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

// ------------------------------------------------------------------ router --

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
#pragma unroll
    for (int w = 1; w < kRouterWarps; ++w) {
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

// -------------------------------------------------------------- the choice --

struct Choice {
  uint16_t expert[kPairs];
  float weight[kPairs];
  uint16_t list[kPairs];             // pairs token * k + j, those of an expert together
  uint16_t active[GE_MOE_MAX_EXPERTS];
  uint16_t count[GE_MOE_MAX_EXPERTS];
  int32_t begin[GE_MOE_MAX_EXPERTS];
  int32_t n_active;
  int32_t counter[GE_MOE_MAX_EXPERTS];
};

// a key in two floats; a larger one first, then the lower index
struct Key {
  float hi, lo;
  int at;
  __device__ __forceinline__ bool before(const Key &o) const {
    return hi > o.hi || (hi == o.hi && (lo > o.lo || (lo == o.lo && at < o.at)));
  }
};

constexpr int kLaneExperts = GE_MOE_MAX_EXPERTS / 32;

// One warp, one token: the k best experts and their weights.
__device__ void choose(const MoeParams &p, int t, Choice &c, bool say) {
  const int lane = threadIdx.x & 31;
  const int mine = (p.E + 31) / 32;
  const float2 *l = p.logits + int64_t(t) * p.E;
  constexpr float kNone = -INFINITY;
  float hi[kLaneExperts], lo[kLaneExperts];
  float top = kNone;
  // (a NaN is no key; its weight is NaN all the same)
#pragma unroll
  for (int i = 0; i < kLaneExperts; ++i) {
    hi[i] = lo[i] = kNone;
    if (i >= mine) continue;
    const int e = i * 32 + lane;
    if (e < p.E) {
      const float2 v = __ldcg(l + e);
      hi[i] = v.x == v.x ? v.x : kNone;
      lo[i] = v.x == v.x ? v.y : 0.f;
      top = fmaxf(top, hi[i]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f;
  if (p.score == GE_SCORE_SOFTMAX) {
    for (int e = lane; e < p.E; e += 32) {
      const float2 v = __ldcg(l + e);
      sum += expf((v.x - top) + v.y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  auto score = [&](float2 v) {
    if (p.score == GE_SCORE_SOFTMAX) return expf((v.x - top) + v.y) / sum;
    return 1.f / (1.f + expf(-v.x) * (1.f - v.y));
  };
  Key best;
  auto find = [&]() {  // the best of all lanes' keys, which is taken away
    best = Key{kNone, kNone, 1 << 30};
#pragma unroll
    for (int i = 0; i < kLaneExperts; ++i) {
      if (i >= mine) continue;
      const Key o{hi[i], lo[i], i * 32 + lane};
      if (o.before(best)) best = o;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Key k{__shfl_xor_sync(0xffffffffu, best.hi, o), __shfl_xor_sync(0xffffffffu, best.lo, o),
                  __shfl_xor_sync(0xffffffffu, best.at, o)};
      if (k.before(best)) best = k;
    }
#pragma unroll
    for (int i = 0; i < kLaneExperts; ++i)
      if (i < mine && i * 32 + lane == best.at) hi[i] = lo[i] = kNone;
  };
  if (p.bias) {
    auto keys = [&](bool exact, double all) {
#pragma unroll
      for (int i = 0; i < kLaneExperts; ++i) {
        hi[i] = lo[i] = kNone;
        const int e = i * 32 + lane;
        if (i >= mine || e >= p.E) continue;
        const float2 v = __ldcg(l + e);
        const float b = __ldg(p.bias + e);
        double key;
        if (exact) {
          const double x = double(v.x) + double(v.y);
          key = (p.score == GE_SCORE_SOFTMAX ? exp(x - double(top)) / all : 1.0 / (1.0 + exp(-x))) + double(b);
          hi[i] = static_cast<float>(key);
          lo[i] = static_cast<float>(key - double(hi[i]));
          if (!isfinite(hi[i])) lo[i] = 0.f;
        } else {
          hi[i] = score(v) + b;
          lo[i] = 0.f;
        }
        if (!(hi[i] == hi[i])) hi[i] = kNone, lo[i] = 0.f;
      }
    };
    // Scores in fp32 are off by a few 1e-7 of themselves: where two of the k + 1 best lie closer than
    // that, all are computed again in 64 bits, which the GPU does slowly.
    keys(false, 0.0);
    bool close = false;
    float last = INFINITY;
    for (int j = 0; j <= p.k && j < p.E; ++j) {
      find();
      close = close || last - best.hi <= 2e-6f * fmaxf(1.f, fabsf(best.hi));
      last = best.hi;
    }
    double all = 0.0;
    if (close && p.score == GE_SCORE_SOFTMAX) {
      for (int e = lane; e < p.E; e += 32) {
        const float2 v = __ldcg(l + e);
        all += exp((double(v.x) - double(top)) + double(v.y));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    keys(close, all);
  }
  float chosen = 0.f, total = 0.f;  // lane j keeps the j-th expert's
  int expert = 0;
  for (int j = 0; j < p.k; ++j) {
    find();
    const float w = score(__ldcg(l + best.at));
    total += w;
    if (lane == j) {
      chosen = w;
      expert = best.at;
    }
  }
  if (lane < p.k) {
    const float w = (p.renormalise ? chosen / total : chosen) * p.route_scale;
    c.expert[t * p.k + lane] = static_cast<uint16_t>(expert);
    c.weight[t * p.k + lane] = w;
    if (say && p.index) p.index[t * p.k + lane] = expert;
    if (say && p.weight) p.weight[t * p.k + lane] = w;
  }
}

// The experts that some token chose, and each one's pairs.
__device__ void make_lists(const MoeParams &p, Choice &c) {
  const int pairs = p.T * p.k;
  for (int e = threadIdx.x; e < p.E; e += kThreads) c.counter[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kThreads) atomicAdd(&c.counter[c.expert[i]], 1);
  __syncthreads();
  if (threadIdx.x < 32) {
    int n = 0, at = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int k = e < p.E ? c.counter[e] : 0;
      const uint32_t some = __ballot_sync(0xffffffffu, k > 0);
      int before = k;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (static_cast<int>(threadIdx.x) >= o) before += v;
      }
      if (k > 0) {
        const int a = n + __popc(some & ((1u << threadIdx.x) - 1u));
        c.active[a] = static_cast<uint16_t>(e);
        c.count[a] = static_cast<uint16_t>(k);
        c.begin[a] = at + before - k;
      }
      if (e < p.E) c.counter[e] = at + before - k;
      n += __popc(some);
      at += __shfl_sync(0xffffffffu, before, 31);
    }
    if (threadIdx.x == 0) c.n_active = n;
  }
  __syncthreads();
  // (an expert's pairs in any order: each has a column of its own)
  for (int i = threadIdx.x; i < pairs; i += kThreads) c.list[atomicAdd(&c.counter[c.expert[i]], 1)] = static_cast<uint16_t>(i);
  __syncthreads();
}

// ---------------------------------------------------------------- products --

template <int XT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (XT == GE_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// h: written by other CTAs of this launch
__device__ __forceinline__ uint4 load_shared(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// two 8-bit floats as two values of type XT (exact)
template <int XT, int WT>
__device__ __forceinline__ uint32_t widen(uint16_t v) {
  uint32_t h;
  if constexpr (WT == GE_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(v));
  if constexpr (XT == GE_F16) return h;
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return pack16(true, f.x, f.y);
}

// acc[tile][..] += a stage's rows (16) x tokens (8 per tile)^T over this warp's columns of the stage, which are
// `first` and up of the whole; `bytes` of each row exist.  `from[n]`: this lane's token of tile n
// (nullptr: zeros); LO: and `rest` elements further what their rounding left.  8-bit weights: scales of this warp's first
// 128 columns at s_lo and s_hi, of the next ld_s further.
template <int XT, int WT, int NT, bool LO>
__device__ __forceinline__ void consume(float (&acc)[NT][4], const uint8_t *stage, int first, int bytes, const uint16_t *const (&from)[NT],
                                        int64_t rest, const float *s_lo, const float *s_hi, int64_t ld_s, int warp, int lane) {
  constexpr bool k8 = WT == GE_E4M3 || WT == GE_E5M2;
  constexpr int kPer = k8 ? 16 : 8;                          // columns of a lane's 16 bytes
  constexpr int kSteps = kSegment / 64 / kWarps;             // of 64 bytes
  constexpr int kStepsOfBlock = k8 ? kBlock / 64 : NT <= 4 ? kSteps : 1;  // whose weights are held at a time
  const int g = lane >> 2, q = lane & 3;
  const int at = warp * kSteps * 64;
  if (at >= bytes) return;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i0 = 0; i0 < kSteps; i0 += kStepsOfBlock) {
    if (at + i0 * 64 >= bytes) break;
    // the weights of a block, or of a step
    uint32_t x0[kStepsOfBlock][kPer / 2], x1[kStepsOfBlock][kPer / 2];
    float s0 = 0.f, s1 = 0.f;
    if constexpr (k8) {
      s0 = __ldg(s_lo + i0 / kStepsOfBlock * ld_s);
      s1 = __ldg(s_hi + i0 / kStepsOfBlock * ld_s);
    }
#pragma unroll
    for (int i = 0; i < kStepsOfBlock; ++i) {
      const int byte = at + (i0 + i) * 64 + q * 16;
      const bool on = byte < bytes;
      const uint4 w0 = on ? *reinterpret_cast<const uint4 *>(stage + g * kPitch + byte) : zero;
      const uint4 w1 = on ? *reinterpret_cast<const uint4 *>(stage + (g + 8) * kPitch + byte) : zero;
      if constexpr (k8) {
        const uint32_t y0[4] = {w0.x, w0.y, w0.z, w0.w}, y1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x0[i][2 * j] = widen<XT, WT>(static_cast<uint16_t>(y0[j]));
          x0[i][2 * j + 1] = widen<XT, WT>(static_cast<uint16_t>(y0[j] >> 16));
          x1[i][2 * j] = widen<XT, WT>(static_cast<uint16_t>(y1[j]));
          x1[i][2 * j + 1] = widen<XT, WT>(static_cast<uint16_t>(y1[j] >> 16));
        }
      } else {
        x0[i][0] = w0.x, x0[i][1] = w0.y, x0[i][2] = w0.z, x0[i][3] = w0.w;
        x1[i][0] = w1.x, x1[i][1] = w1.y, x1[i][2] = w1.z, x1[i][3] = w1.w;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      float(&d)[4] = k8 ? sum : acc[n];
#pragma unroll
      for (int i = 0; i < kStepsOfBlock; ++i) {
        const bool on = at + (i0 + i) * 64 + q * 16 < bytes;
        const int col = first + (at + (i0 + i) * 64) / (k8 ? 1 : 2) + q * kPer;
#pragma unroll
        for (int l = 0; l < (LO ? 2 : 1); ++l) {
#pragma unroll
          for (int u = 0; u < kPer / 8; ++u) {
            uint4 b = zero;
            if (from[n] && on) {
              const uint16_t *s = from[n] + (l ? rest : 0) + col + 8 * u;
              b = LO ? load_shared(s) : __ldg(reinterpret_cast<const uint4 *>(s));
            }
            mma<XT>(d, x0[i][4 * u], x1[i][4 * u], x0[i][4 * u + 1], x1[i][4 * u + 1], b.x, b.y);
            mma<XT>(d, x0[i][4 * u + 2], x1[i][4 * u + 2], x0[i][4 * u + 3], x1[i][4 * u + 3], b.z, b.w);
          }
        }
      }
      if constexpr (k8) {
        acc[n][0] = fmaf(sum[0], s0, acc[n][0]);
        acc[n][1] = fmaf(sum[1], s0, acc[n][1]);
        acc[n][2] = fmaf(sum[2], s1, acc[n][2]);
        acc[n][3] = fmaf(sum[3], s1, acc[n][3]);
      }
    }
  }
}

// The warps' sums of some tokens, side by side for whoever adds them: [warp][token][row]
struct Sums {
  float v[kWarps][kRoundTiles * kTile][16];
};

__device__ __forceinline__ float total(const Sums &s, int token, int row) {
  float v = s.v[0][token][row];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += s.v[w][token][row];
  return v;
}

__device__ __forceinline__ float activate(int act, float g) {
  if (act == GE_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  if (act == GE_RELU) return g > 0.f ? g : (g == g ? 0.f : g);
  return g / (1.f + expf(-g));
}

template <int XT>
__device__ __forceinline__ float round_trip(uint16_t v) {
  if constexpr (XT == GE_BF16) return __uint_as_float(uint32_t(v) << 16);
  else return __half2float(__ushort_as_half(v));
}

struct Shared {
  Choice c;
  Sums sums[2];
  alignas(8) uint64_t full[kStages], empty[kStages];          // stages of the ring
  alignas(8) uint64_t taken[kQueue], ready[kQueue], out[kQueue], free[kQueue];  // a unit: named, its h there, written, forgotten
  uint32_t unit[kQueue];
  volatile uint32_t quit;
  alignas(128) uint8_t ring[kStages][16 * kPitch];
};

constexpr uint32_t kNoUnit = 0xffffffffu;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t add_acq_rel(uint32_t *p, uint32_t by) {
  uint32_t v;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(v) : "l"(p), "r"(by) : "memory");
  return v;
}

__device__ __forceinline__ void add_release(uint32_t *p, uint32_t by) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(by) : "memory");
}

__device__ void give_up(const MoeParams &p, Shared &sh) {
  if (atomicCAS(p.status, 0u, static_cast<uint32_t>(GE_ERR_TIMEOUT)) == 0u) {
    p.status[1] = 0;
    p.status[2] = blockIdx.x;
  }
  atomicExch(&p.head->abort, 1u);
  sh.quit = 1u;
}

// Waits within a CTA: false where it gives up.  (They last as long as another CTA's h does, and four times the
// time a watcher waits for that at most.)
__device__ __forceinline__ bool wait_bar(const MoeParams &p, Shared &sh, const uint64_t &bar, uint32_t parity) {
  const uint32_t b = smem_u32(&bar);
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(b, parity, 20000u)) return true;
    if (sh.quit) return false;
    if (globaltimer_ns() - t0 > 4 * p.timeout_ns) {
      give_up(p, sh);
      return false;
    }
  }
}

// an expert's h: false where the time ran out or another CTA's did
__device__ bool wait_for(const MoeParams &p, Shared &sh, const uint32_t *counter, uint32_t want) {
  if (load_acquire(counter) >= want) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (load_acquire(counter) >= want) return true;
    if (load_acquire(&p.head->abort)) {
      sh.quit = 1u;
      return false;
    }
    if (globaltimer_ns() - t0 > p.timeout_ns) {
      give_up(p, sh);
      return false;
    }
    __nanosleep(64);
  }
}

// A unit of work: `a` the active expert, `col` its first column of h or of y.
struct Unit {
  int a, col;
  bool up;
};

struct Units {
  uint32_t up_cols, down_cols, n_up, n_all;
  __device__ __forceinline__ Units(const MoeParams &p, int n_active) {
    up_cols = p.F / kUpCols;
    down_cols = (p.D + kDownCols - 1) / kDownCols;
    n_up = n_active * up_cols;
    n_all = n_up + n_active * down_cols;
  }
  __device__ __forceinline__ Unit of(uint32_t u) const {
    Unit r;
    r.up = u < n_up;
    const uint32_t v = r.up ? u : u - n_up, per = r.up ? up_cols : down_cols;
    r.a = v / per;
    r.col = (v - r.a * per) * (r.up ? kUpCols : kDownCols);
    return r;
  }
};

// A position in a ring of N.
template <int N>
struct Turn {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// The consumers' part of a unit with up to 8 NT tokens; false where a wait gave up.
template <int XT, int WT, int NT, bool UP>
__device__ bool do_unit(const MoeParams &p, Shared &sh, const Unit &u, Turn<kStages> &st, int &round) {
  constexpr bool k8 = WT == GE_E4M3 || WT == GE_E5M2;
  constexpr int ws = k8 ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const Choice &c = sh.c;
  const int e = c.active[u.a], n = c.count[u.a];
  const uint16_t *list = c.list + c.begin[u.a];
  const int K = UP ? p.D : p.F, segments = (K * ws + kSegment - 1) / kSegment;
  const int64_t rest = int64_t(p.T) * p.k * p.F;
  const float *s_lo = nullptr, *s_hi = nullptr;
  int64_t ld_s = 0;
  if constexpr (k8) {
    ld_s = ((UP ? 2 * p.F : p.D) + kBlock - 1) / kBlock;
    const float *f = (UP ? p.s_up : p.s_down) + int64_t(e) * ld_s * ((K + kBlock - 1) / kBlock) + warp * (kSegment / kWarps / kBlock) * ld_s;
    s_lo = f + u.col / kBlock;
    s_hi = f + (UP ? p.F + u.col : u.col) / kBlock;
  }
  const uint16_t *from[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int at = i * kTile + g;
    from[i] = at >= n ? nullptr : UP ? static_cast<const uint16_t *>(p.x) + int64_t(list[at] / p.k) * p.ldx : p.h + int64_t(list[at]) * p.F;
  }
  float acc[NT][4] = {};
  for (int j = 0; j < segments; ++j) {
    if (!__all_sync(0xffffffffu, wait_bar(p, sh, sh.full[st.at], st.phase))) return false;
    consume<XT, WT, NT, !UP>(acc, sh.ring[st.at], j * (kSegment / ws), min(kSegment, K * ws - j * kSegment), from, rest, s_lo, s_hi, ld_s, warp,
                             lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st.at]));
    st.next();
    if constexpr (k8) {
      s_lo += kSegment / kBlock * ld_s;
      s_hi += kSegment / kBlock * ld_s;
    }
  }
  // the warps' sums, 16 tokens at a time (a buffer's last readers have passed the barrier of the round between)
#pragma unroll
  for (int r = 0; r < NT; r += kRoundTiles) {
    if (r * kTile >= n) break;
    Sums &s = sh.sums[round++ & 1];
#pragma unroll
    for (int i = 0; i < kRoundTiles; ++i) {
      if (r + i >= NT) break;
      s.v[warp][i * kTile + 2 * q][g] = acc[r + i][0];
      s.v[warp][i * kTile + 2 * q + 1][g] = acc[r + i][1];
      s.v[warp][i * kTile + 2 * q][g + 8] = acc[r + i][2];
      s.v[warp][i * kTile + 2 * q + 1][g + 8] = acc[r + i][3];
    }
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    const int some = min(n - r * kTile, kRoundTiles * kTile);
    const uint16_t *of = list + r * kTile;
    if constexpr (UP) {
      for (int i = threadIdx.x; i < some * kUpCols; i += 32 * kWarps) {
        const int token = i / kUpCols, row = i % kUpCols;
        const float v = activate(p.act, total(s, token, row)) * total(s, token, row + 8);
        const uint16_t hi = static_cast<uint16_t>(pack16(XT == GE_BF16, v, 0.f));
        const float left = v - round_trip<XT>(hi);
        uint16_t *h = p.h + int64_t(of[token]) * p.F + u.col + row;
        h[0] = hi;
        // (nothing is left of an infinity)
        h[rest] = isfinite(left) ? static_cast<uint16_t>(pack16(XT == GE_BF16, left, 0.f)) : 0;
      }
    } else {
      for (int i = threadIdx.x; i < some * kDownCols; i += 32 * kWarps) {
        const int token = i / kDownCols, row = i % kDownCols;
        if (u.col + row < p.D) p.part[int64_t(of[token]) * p.D + u.col + row] = total(s, token, row) * c.weight[of[token]];
      }
    }
  }
  return true;
}

template <int XT, int WT, bool UP>
__device__ bool any_unit(const MoeParams &p, Shared &sh, const Unit &u, Turn<kStages> &st, int &round) {
  const int n = sh.c.count[u.a];
  if (n <= kTile) return do_unit<XT, WT, 1, UP>(p, sh, u, st, round);
  if (n <= 2 * kTile) return do_unit<XT, WT, 2, UP>(p, sh, u, st, round);
  if (n <= 4 * kTile) return do_unit<XT, WT, 4, UP>(p, sh, u, st, round);
  return do_unit<XT, WT, GE_MOE_MAX_TOKENS / kTile, UP>(p, sh, u, st, round);
}

// y's 16 columns of all tokens: a lane adds 8 columns of a token, in the order of its choice
template <int XT>
__device__ void add_shares(const MoeParams &p, int col) {
  for (int i = threadIdx.x & 31; i < p.T * 2; i += 32) {
    const int t = i >> 1, d0 = col + (i & 1) * 8;
    if (d0 >= p.D) continue;
    float v[8] = {};
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
      const float4 *f = reinterpret_cast<const float4 *>(p.part + (int64_t(t) * p.k + j) * p.D + d0);
      const float4 x = __ldcg(f), y = __ldcg(f + 1);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack16(XT == GE_BF16, v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + int64_t(t) * p.ldy + d0) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int XT, int WT>
__global__ void __launch_bounds__(kThreads, 1) moe_experts_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  Shared &sh = *reinterpret_cast<Shared *>(smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u));
  constexpr int ws = WT == GE_E4M3 || WT == GE_E5M2 ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), kWarps);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(smem_u32(&sh.taken[i]), 1);
      mbar_init(smem_u32(&sh.ready[i]), 1);
      mbar_init(smem_u32(&sh.out[i]), kWarps);
      mbar_init(smem_u32(&sh.free[i]), 1);
    }
    sh.quit = 0u;
    fence_mbarrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  for (int t = warp; t < p.T; t += kThreads / 32) choose(p, t, sh.c, blockIdx.x == 0);
  __syncthreads();
  make_lists(p, sh.c);
  const Units units(p, sh.c.n_active);
  Turn<kQueue> slot;
  Turn<kStages> st;

  if (warp == kProducer) {
    int filled = 0;
    bool ok = true;
    while (ok) {
      uint32_t t = 0;
      if (lane == 0) t = atomicAdd(&p.head->ticket, 1u);
      t = __shfl_sync(0xffffffffu, t, 0);
      const bool last = t >= units.n_all;
      ok = __all_sync(0xffffffffu, wait_bar(p, sh, sh.free[slot.at], slot.phase ^ 1u));
      if (!ok) break;
      if (lane == 0) {
        sh.unit[slot.at] = last ? kNoUnit : t;
        mbar_arrive(smem_u32(&sh.taken[slot.at]));
      }
      slot.next();
      if (last) break;
      const Unit u = units.of(t);
      const int e = sh.c.active[u.a], K = u.up ? p.D : p.F;
      // this lane's row
      const int64_t r = u.up ? int64_t(e) * 2 * p.F + u.col + (lane & 7) + (lane & 8 ? p.F : 0) : int64_t(e) * p.D + u.col + (lane & 15);
      const uint8_t *row = static_cast<const uint8_t *>(u.up ? p.w_up : p.w_down) + r * K * ws;
      const int rows = u.up ? 16 : min(16, p.D - u.col);
      for (int at = 0; at < K * ws; at += kSegment) {
        ok = __all_sync(0xffffffffu, wait_bar(p, sh, sh.empty[st.at], st.phase ^ 1u));
        if (!ok) break;
        const uint32_t bytes = min(kSegment, K * ws - at), full = smem_u32(&sh.full[st.at]);
        if (lane == 0) mbar_arrive_expect_tx(full, bytes * rows);
        __syncwarp();
        if (lane < rows) bulk_load(smem_u32(sh.ring[st.at] + lane * kPitch), row + at, bytes, full);
        st.next();
        ++filled;
      }
    }
    if (!ok)  // what is on its way lands before the CTA's shared memory is another's
      for (int f = max(0, filled - kStages); f < filled; ++f) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&sh.full[f % kStages]), static_cast<uint32_t>(f / kStages) & 1u))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
      }
  } else if (warp == kWatcher) {
    if (lane == 0)
      for (;;) {
        if (!wait_bar(p, sh, sh.taken[slot.at], slot.phase)) break;
        const uint32_t t = sh.unit[slot.at];
        if (t != kNoUnit && t >= units.n_up && !wait_for(p, sh, &p.done[sh.c.active[units.of(t).a]], units.up_cols)) break;
        mbar_arrive(smem_u32(&sh.ready[slot.at]));
        slot.next();
        if (t == kNoUnit) break;
      }
  } else if (warp == kFinisher) {
    for (;;) {
      if (!__all_sync(0xffffffffu, wait_bar(p, sh, sh.out[slot.at], slot.phase))) break;
      const uint32_t t = sh.unit[slot.at];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.free[slot.at]));
      slot.next();
      if (t == kNoUnit) break;
      const Unit u = units.of(t);
      if (u.up) {
        if (lane == 0 && !(t == 0 && (p.debug_flags & GE_DEBUG_SKIP_FIRST_LOAD))) add_release(&p.done[sh.c.active[u.a]], 1u);
      } else {
        uint32_t before = 0;
        if (lane == 0) before = add_acq_rel(&p.shares[u.col / kDownCols], 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == static_cast<uint32_t>(sh.c.n_active) - 1u) add_shares<XT>(p, u.col);
      }
    }
  } else {
    int round = 0;
    for (;;) {
      if (!__all_sync(0xffffffffu, wait_bar(p, sh, sh.ready[slot.at], slot.phase))) break;
      const uint32_t t = sh.unit[slot.at];
      if (t != kNoUnit) {
        const Unit u = units.of(t);
        if (!(u.up ? any_unit<XT, WT, true>(p, sh, u, st, round) : any_unit<XT, WT, false>(p, sh, u, st, round))) break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.out[slot.at]));
      slot.next();
      if (t == kNoUnit) break;
    }
  }
}

constexpr int kSmem = static_cast<int>(sizeof(Shared)) + 128;

template <int XT>
const void *experts(int wt) {
  switch (wt) {
    case GE_E4M3: return reinterpret_cast<const void *>(moe_experts_kernel<XT, GE_E4M3>);
    case GE_E5M2: return reinterpret_cast<const void *>(moe_experts_kernel<XT, GE_E5M2>);
    default: return reinterpret_cast<const void *>(moe_experts_kernel<XT, XT>);
  }
}

}  // namespace

struct gemm_epi_moe_plan {
  MoeParams p;
  const void *router, *experts;
  int grid;
  bool k8;
};

namespace {

struct Space {
  size_t done, shares, logits, h, part, bytes;
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
  pl->experts = d.x == GE_BF16 ? experts<GE_BF16>(d.w) : experts<GE_F16>(d.w);
  const bool f32 = d.router == GE_F32;
  if (d.x == GE_BF16)
    pl->router = f32 ? reinterpret_cast<const void *>(moe_router_kernel<GE_BF16, true>)
                     : reinterpret_cast<const void *>(moe_router_kernel<GE_BF16, false>);
  else
    pl->router = f32 ? reinterpret_cast<const void *>(moe_router_kernel<GE_F16, true>)
                     : reinterpret_cast<const void *>(moe_router_kernel<GE_F16, false>);
  int per_sm = 0;
  if (!p.status || cudaFuncSetAttribute(pl->experts, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, pl->experts, kThreads, kSmem) != cudaSuccess || per_sm < 1) {
    cudaGetLastError();
    delete pl;
    return GE_ERR_CUDA;
  }
  const int64_t most = std::min<int64_t>(E, T * k) * (F / kUpCols + ceil_div(D, kDownCols));
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
  p.h = reinterpret_cast<uint16_t *>(ws + s.h);
  p.part = reinterpret_cast<float *>(ws + s.part);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *args[] = {&p};
  if (launch_pdl(pl->router, dim3(static_cast<unsigned>(p.E), static_cast<unsigned>(ceil_div(p.T, kRouterTokens))),
                 dim3(32 * kRouterWarps), 0, args, st) != cudaSuccess)
    return GE_ERR_CUDA;
  return launch_pdl(pl->experts, dim3(static_cast<unsigned>(pl->grid)), dim3(kThreads), kSmem, args, st) == cudaSuccess ? GE_OK
                                                                                                                   : GE_ERR_CUDA;
}

}  // extern "C"
