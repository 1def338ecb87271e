// moe_choice.cuh -- a token's experts and their weights, from its logits.
#pragma once

#include <stdint.h>

#include "moe.h"

namespace ge {

// floats as integers in the same order
__device__ __forceinline__ int ordered(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7fffffff);
}

// What an expert is chosen by, two floats, as integers of the same order; an upper one of 0 is below all.
__device__ __forceinline__ uint32_t key_of(float f) { return static_cast<uint32_t>(ordered(f + 0.f)) ^ 0x80000000u; }  // (-0 is 0)
__device__ __forceinline__ float of_key(uint32_t k) { return __int_as_float(ordered(__int_as_float(static_cast<int>(k ^ 0x80000000u)))); }

__device__ __forceinline__ float sigmoid_of(float2 v) {  // v.y: what the rounding of the argument left
  const float e = expf(-fabsf(v.x)) * (v.x < 0.f ? 1.f + v.y : 1.f - v.y);
  return (v.x < 0.f ? e : 1.f) / (1.f + e);
}

// exp(v - m).  A difference of 16 is off by up to 2^-20, and so is then its exponential, by that much of itself: what the
// rounding left is kept, as for v (infinities and NaN have no remainder).
__device__ __forceinline__ float exp_from(float2 v, float m) {
  const float d = __fsub_rn(v.x, m), b = __fsub_rn(d, v.x);
  const float left = __fadd_rn(__fsub_rn(v.x, __fsub_rn(d, b)), __fsub_rn(-m, b));
  return expf(d) * (isfinite(d) ? 1.f + (left + v.y) : 1.f);
}

struct ChoiceSpace {  // a warp's
  float2 logits[GE_MOE_MAX_EXPERTS];
  alignas(16) uint32_t upper[GE_MOE_MAX_EXPERTS];
  uint32_t lower[GE_MOE_MAX_EXPERTS];
  uint32_t best[32];   // upper keys of the chosen
  int32_t which[32];
  __device__ __forceinline__ void put(int e, float hi, float lo) {  // a NaN counts as -infinity
    upper[e] = key_of(hi == hi ? hi : -INFINITY);
    lower[e] = key_of(isfinite(hi) ? lo : 0.f);
  }
};

// The `some` best of up to 32 N experts, by how many are above each: a single warp's time is what it issues one after
// another, and these comparisons do not wait for each other.  (For more than 64 experts they are too many: 64 tokens'
// choice among 128 took 44 us instead of 27.)  Upper keys alone: false, with nothing stored, where one of the best is equal
// to another of them or to one that is left out.
template <int N>
__device__ __forceinline__ bool rank(int E, int some, ChoiceSpace &s) {
  const int lane = threadIdx.x & 31;
  uint32_t mine[N];
  int above[N] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) mine[i] = i * 32 + lane < E ? s.upper[i * 32 + lane] : 0;
  for (int e = E + lane; e < (E + 3) / 4 * 4; e += 32) s.upper[e] = 0;
  __syncwarp();
#pragma unroll 2
  for (int e = 0; e < E; e += 4) {
    const uint4 o = *reinterpret_cast<const uint4 *>(&s.upper[e]);
#pragma unroll
    for (int i = 0; i < N; ++i) above[i] += (o.x > mine[i]) + (o.y > mine[i]) + (o.z > mine[i]) + (o.w > mine[i]);
  }
  // How many have a place, above the sum of 2^place (64 times 2^16 at most).  Groups of equal keys g at place a add g to the
  // number and g 2^a to the sum; as many as wanted with a sum of 2^some - 1 are one for each place.
  constexpr uint32_t kOne = 1u << 25;
  uint32_t places = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (mine[i] != 0 && above[i] < some) places += kOne + (1u << above[i]);
  if (__reduce_add_sync(0xffffffffu, places) != some * kOne + (1u << some) - 1u) return false;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (mine[i] != 0 && above[i] < some) {
      s.best[above[i]] = mine[i];
      s.which[above[i]] = i * 32 + lane;
    }
  return true;
}

// The `some` best experts in order, of equal keys the lower index first; whether two neighbours' upper keys are close.
__device__ __forceinline__ bool find_best(int E, int some, ChoiceSpace &s) {
  const int lane = threadIdx.x & 31;
  const bool ranked = E <= 32 ? rank<1>(E, some, s) : E <= 64 ? rank<2>(E, some, s) : false;
  if (!ranked) {
    uint32_t hi, lo;  // this lane's best, found again when it has been taken
    int at;
    auto look = [&]() {
      hi = lo = 0;
      at = E;
#pragma unroll 4
      for (int e = lane; e < E; e += 32) {
        const uint32_t h = s.upper[e], w = s.lower[e];
        if (h > hi || (h == hi && h != 0 && w > lo)) hi = h, lo = w, at = e;
      }
    };
    look();
#pragma unroll 1
    for (int j = 0; j < some; ++j) {
      const uint32_t most = __reduce_max_sync(0xffffffffu, hi), rest = __reduce_max_sync(0xffffffffu, hi == most ? lo : 0u);
      const int e = __reduce_min_sync(0xffffffffu, hi == most && lo == rest ? at : E);
      if (at == e) {
        s.best[j] = most;
        s.which[j] = e;
        s.upper[e] = 0;
        look();
      }
      __syncwarp();
    }
  }
  __syncwarp();
  const float now = lane < some ? of_key(s.best[lane]) : 0.f;
  const float next = __shfl_down_sync(0xffffffffu, now, 1);
  return __any_sync(0xffffffffu, lane + 1 < some && now - next <= 2e-6f * fmaxf(1.f, fabsf(now)));
}

// One warp, one token: the k best experts and their weights.  This may run once in every CTA, so its code is short.
// (Unrolled over keys in registers it took 8 us for one token and 124 us for 64 with 128 experts.)
static __device__ __noinline__ void choose(const MoeParams &p, int t, uint16_t *experts, float *weights, ChoiceSpace &s, bool say) {
  const int lane = threadIdx.x & 31;
  const bool softmax = p.score == GE_SCORE_SOFTMAX;
  const float2 *l = s.logits;
  float top = -INFINITY;
#pragma unroll 4
  for (int e = lane; e < p.E; e += 32) {
    const float2 v = __ldcg(p.logits + int64_t(t) * p.E + e);
    s.logits[e] = v;
    if (!p.bias) s.put(e, v.x, v.y);
    top = fmaxf(top, v.x);
  }
  float sum = 0.f;
  if (softmax && (p.bias || !p.renormalise)) {
    top = __int_as_float(ordered(__int_as_float(__reduce_max_sync(0xffffffffu, ordered(top)))));
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) sum += expf((l[e].x - top) + l[e].y);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (p.bias) {
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
      const float2 v = l[e];
      s.put(e, (softmax ? expf((v.x - top) + v.y) / sum : sigmoid_of(v)) + __ldg(p.bias + e), 0.f);
    }
    __syncwarp();
    // Scores in fp32 are off by a few 1e-7 of themselves: where two of the k + 1 best lie closer than
    // that, all are computed again in 64 bits, which the GPU does slowly.
    if (find_best(p.E, min(p.k + 1, p.E), s)) {
      double all = 0.0;
      if (softmax) {
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) all += exp((double(l[e].x) - double(top)) + double(l[e].y));
#pragma unroll 1
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      }
#pragma unroll 1
      for (int e = lane; e < p.E; e += 32) {
        const double x = double(l[e].x) + double(l[e].y), ex = exp(softmax ? x - double(top) : -x);
        const double score = (softmax ? ex / all : 1.0 / (1.0 + ex)) + double(__ldg(p.bias + e));
        const float hi = static_cast<float>(score);
        s.put(e, hi, static_cast<float>(score - double(hi)));
      }
      __syncwarp();
      find_best(p.E, p.k, s);
    }
  } else {
    __syncwarp();
    find_best(p.E, p.k, s);
  }
  // lane j: the j-th expert
  const int expert = lane < p.k ? s.which[lane] : 0;
  const float2 v = lane < p.k ? l[expert] : make_float2(-INFINITY, 0.f);
  float w;
  if (p.renormalise) {
    // what cancels is left out, so that scores of nothing but far experts do not vanish: softmax's sum, and
    // the largest one's exponential where all are small
    const float m = __int_as_float(ordered(__int_as_float(__reduce_max_sync(0xffffffffu, ordered(v.x == v.x ? v.x : -INFINITY)))));
    w = softmax || m < 0.f ? exp_from(v, m) : 0.f;
    if (!softmax) w = m < 0.f ? w / (1.f + expf(v.x)) : sigmoid_of(v);
    float total = lane < p.k ? w : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    w /= total;
  } else {
    w = softmax ? exp_from(v, top) / sum : sigmoid_of(v);
  }
  if (lane < p.k) {
    w *= p.route_scale;
    experts[t * p.k + lane] = static_cast<uint16_t>(expert);
    weights[t * p.k + lane] = w;
    if (say && p.index) p.index[t * p.k + lane] = expert;
    if (say && p.weight) p.weight[t * p.k + lane] = w;
  }
  __syncwarp();
}

}  // namespace ge
