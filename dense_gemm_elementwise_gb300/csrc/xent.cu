// xent.cu -- the vocabulary loss and its gradients (gemm_epi_xent_*): plan,
// launches, and the small kernels around the products of xent_kernel.cuh.
//
//   pack     which rows take part (their target exists), in their order: hidden
//            states, targets and weights side by side, zero rows up to the next
//            k-block; ignored rows get loss and lse 0
//   X_KEEP   (X_STATS for fp16) logits -> per row and column range: maximum, sum, target's logit; of
//            the first piece of the vocabulary also the logits, in 16 bits
//   finish   joins the ranges: lse, loss, total; what the gradients need per row
//   per piece of the vocabulary:
//     convert / X_DLOGIT  dl of the piece, from what was kept / from the product again
//     X_OUT    dW rows of the piece = dl^T @ H
//     X_PART   dH += dl @ W, fp32
//   spread   dH slices added in order, rounded, back to the rows' places
//
// A loss alone is X_STATS and finish, after pack where that can save tiles.
// How many rows take part stays on the device.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "gemm_epi.h"
#include "host.h"
#include "ptx.cuh"
#include "xent.cuh"
#include "xent_math.cuh"

using namespace ge;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2Hi = 0.69314718f, kLn2Lo = static_cast<float>(0.69314718055994531 - double(kLn2Hi));

__device__ __forceinline__ int64_t target_of(const void *t, int i32, int64_t i) {
  return i32 ? static_cast<const int32_t *>(t)[i] : static_cast<const int64_t *>(t)[i];
}

// dH's sum over the vocabulary: tiles of m x n, k-blocks, CTAs (pairs), slices at most
struct SplitParams {
  int32_t m, n, n_blk, kb, units, slices;
};

// dH has few tiles for its long sum.  Whole waves of them are left whole; the k-blocks of those
// left over are split so that the slices fill one to four waves of CTAs in the
// least time (in k-blocks of a tile, 0.27 us each: the waves' k-blocks and about six for
// set-up and stores, and the slices' way to memory and back).
__device__ void choose_split(const SplitParams &p, int rows, XentScalars *sc) {
  const int tiles = max(1, (rows + p.m - 1) / p.m) * p.n_blk;
  const int full = tiles / p.units * p.units, rest = tiles - full;
  float best = 0.f;
  int best_kbs = p.kb;
  for (int w = 0; w <= 4 && rest > 0; ++w) {
    const int s = max(1, w == 0 ? 1 : min(min(p.units * w / rest, p.slices), p.kb));
    const int kbs = (p.kb + s - 1) / s, used = (p.kb + kbs - 1) / kbs;
    const int waves = (rest * used + p.units - 1) / p.units;
    const float cost = float(waves) * float(kbs + 6) +
                       float(used) * float(rest) * float(p.m * p.n) * (8.f / (6.5e6f * 0.27f));
    if (w == 0 || cost < best * 0.9f) {
      best = cost;
      best_kbs = kbs;
    }
  }
  sc->rows = rows;
  sc->full = full;
  sc->kb_split = best_kbs;
}

struct PackParams {
  const void *target;
  const float *weight;
  const uint16_t *H;
  uint16_t *Hc;
  float *loss, *lse;
  XentScalars *sc;
  int32_t *index, *place, *gathered;  // row of the r-th taken, its inverse (-1: ignored), targets
  float *gweight;
  int64_t V, ldh, ldc;
  int32_t T, D, i32, rows_per_cta;
  SplitParams split;
};

// Every CTA packs a run of rows.  It counts the rows that take part before its
// own from the targets themselves (they are few bytes and in L2 after the
// first CTA), which costs less than a launch or a chain of CTAs.
constexpr int kPackThreads = 256;
__global__ void __launch_bounds__(kPackThreads) xent_pack_kernel(const __grid_constant__ PackParams p) {
  __shared__ int counts[2][kPackThreads / 32];
  __shared__ int32_t rows[kPackThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t begin = int64_t(blockIdx.x) * p.rows_per_cta, end = min(begin + p.rows_per_cta, int64_t(p.T));
  int before = 0, all = 0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < p.T; i += kPackThreads) {
    const int64_t t = target_of(p.target, p.i32, i);
    const int take = t >= 0 && t < p.V;
    all += take;
    before += i < begin ? take : 0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if (lane == 0) {
    counts[0][warp] = before;
    counts[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kPackThreads / 32; ++w) {
    before += counts[0][w];
    all += counts[1][w];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) choose_split(p.split, all, p.sc);
  auto copy = [&](const uint16_t *src, int64_t r) {  // a warp copies one row, or zeros
    uint16_t *dst = p.Hc + r * p.ldc;
    const int whole = p.D / 8 * 8;
#pragma unroll 4
    for (int c = lane * 8; c < whole; c += 256)
      *reinterpret_cast<uint4 *>(dst + c) = src ? *reinterpret_cast<const uint4 *>(src + c) : make_uint4(0u, 0u, 0u, 0u);
    if (whole + lane < p.D) dst[whole + lane] = src ? src[whole + lane] : uint16_t(0);
  };
  for (int64_t first = begin; first < end; first += kPackThreads) {
    const int64_t i = first + threadIdx.x;
    const int64_t t = i < end ? target_of(p.target, p.i32, i) : -1;
    const bool take = t >= 0 && t < p.V;
    const unsigned vote = __ballot_sync(0xffffffffu, take);
    __syncthreads();
    if (lane == 0) counts[0][warp] = __popc(vote);
    __syncthreads();
    int at = __popc(vote & ((1u << lane) - 1u)), here = 0;
#pragma unroll
    for (int w = 0; w < kPackThreads / 32; ++w) {
      at += w < warp ? counts[0][w] : 0;
      here += counts[0][w];
    }
    if (take) {
      const int r = before + at;
      rows[at] = static_cast<int32_t>(i);
      p.index[r] = static_cast<int32_t>(i);
      p.gathered[r] = static_cast<int32_t>(t);
      p.gweight[r] = p.weight ? p.weight[i] : 1.f;
      p.place[i] = r;
    } else if (i < end) {
      p.place[i] = -1;
      if (p.loss) p.loss[i] = 0.f;
      if (p.lse) p.lse[i] = 0.f;
    }
    __syncthreads();
    // with every row taking part the products read H itself
    for (int k = warp; k < (all < p.T ? here : 0); k += kPackThreads / 32) copy(p.H + rows[k] * p.ldh, before + k);
    before += here;
  }
  if (blockIdx.x == gridDim.x - 1 && all < p.T) {
    const int64_t stop = min(int64_t(p.T), (int64_t(all) + BK - 1) / BK * BK);
    for (int64_t r = all + warp; r < stop; r += kPackThreads / 32) copy(nullptr, r);
  }
}

struct FinishParams {
  const float2 *stats;       // [slots][T]
  const float *at_target;
  const int32_t *index;      // nullptr: rows were not packed, ...
  const float *gweight;
  const void *target;        // ... these say which take part
  const float *weight;
  float *loss, *lse, *total;
  float *lse2;
  float2 *coef;
  float4 *block_sums;        // per block: losses, weights, the largest factor of dl
  XentScalars *sc;
  // rows that were not packed and whose gradients follow: a block per row, which leaves what
  // packing would (the row itself or zeros, its target or -1, its place)
  const uint16_t *H;
  uint16_t *Hc;
  int32_t *gathered, *place;
  int64_t ldh, ldc;
  SplitParams split;
  int64_t V;
  int32_t T, D, i32, slots, row_lanes;  // row_lanes rows per block of 1024 threads
  int32_t mean;
  float z, grad_scale, c;
};

// (maximum, sum of 2^(x - maximum)) of two sets joined
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), off = top == -INFINITY ? 0.f : top;
  return make_float2(top, a.y * exp2f(a.x - off) + b.y * exp2f(b.x - off));
}

__device__ __forceinline__ float3 add_over_warp(float3 v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, s);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, s);
    v.z = fmaxf(v.z, __shfl_xor_sync(0xffffffffu, v.z, s));
  }
  return v;
}

// row_lanes consecutive rows per block; the other threads share each row's
// column ranges.  The last block to finish adds the blocks' sums, as every sum here
// in a tree of fixed shape.  Bound by the latency of its loads and barriers when rows are
// few and by its bytes (8 per row and 64 or 128 columns) when they are many.
__global__ void __launch_bounds__(1024) xent_finish_kernel(const __grid_constant__ FinishParams p) {
  __shared__ float2 pairs[1024];
  __shared__ float4 sums[32];
  __shared__ bool last;
  griddep_wait();
  griddep_launch_dependents();
  const int rows = p.index ? p.sc->rows : p.T;
  const int per = p.row_lanes, lanes = 1024 / per;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = threadIdx.x % per, y = threadIdx.x / per;
  const int r = blockIdx.x * per + x;
  float2 all = make_float2(-INFINITY, 0.f);
  if (r < rows) {
    for (int s = y; s < p.slots; s += 8 * lanes) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = s + i * lanes < p.slots ? p.stats[int64_t(s + i * lanes) * p.T + r] : make_float2(-INFINITY, 0.f);
      float top = all.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, v[i].x);
      const float off = top == -INFINITY ? 0.f : top;
      float sum = all.y * exp2f(all.x - off);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i].y * exp2f(v[i].x - off);
      all = make_float2(top, sum);
    }
  }
  // threads of the same row within a warp, then warp x joins row x's 32 warps
  for (int h = per; h < 32; h <<= 1)
    all = join(all, make_float2(__shfl_xor_sync(0xffffffffu, all.x, h), __shfl_xor_sync(0xffffffffu, all.y, h)));
  if (lane < per) pairs[warp * per + lane] = all;
  __syncthreads();
  float3 sum = make_float3(0.f, 0.f, 0.f);
  if (warp < per) {
    const int row = blockIdx.x * per + warp;
    all = pairs[lane * per + warp];
#pragma unroll
    for (int h = 16; h > 0; h >>= 1)
      all = join(all, make_float2(__shfl_xor_sync(0xffffffffu, all.x, h), __shfl_xor_sync(0xffffffffu, all.y, h)));
    if (lane == 0 && row < rows) {
      int64_t i = row;
      bool take = true;
      float w = 1.f;
      if (p.index) {
        i = p.index[row];
        w = p.gweight[row];
      } else {
        const int64_t t = target_of(p.target, p.i32, i);
        take = t >= 0 && t < p.V;
        if (p.weight) w = p.weight[i];
      }
      if (take) {
        // lse = ln 2 (top + log2 sum), its large part split so that loss loses nothing to it
        const float top = all.x == -INFINITY ? 0.f : all.x, l2 = log2f(all.y);
        const float big = top * kLn2Hi;
        const float rest = fmaf(top, kLn2Hi, -big) + fmaf(top, kLn2Lo, l2 * kLn2Hi);
        const float lse = big + rest;
        const float loss = w * (((big - p.at_target[row]) + rest) + p.z * lse * lse);
        if (p.loss) p.loss[i] = loss;
        if (p.lse) p.lse[i] = lse;
        sum = make_float3(loss, w, 0.f);
        if (p.coef) {
          const float zf = 1.f + 2.f * p.z * lse;
          p.lse2[row] = top + l2;
          p.coef[row] = make_float2(w * zf, w);
          const float b = fabsf(w) * fmaxf(1.f, fabsf(zf));
          sum.z = isfinite(b) ? b : 0.f;
        }
      } else {
        if (p.loss) p.loss[i] = 0.f;
        if (p.lse) p.lse[i] = 0.f;
        if (p.coef) {
          p.lse2[row] = 0.f;
          p.coef[row] = make_float2(0.f, 0.f);
        }
      }
      if (p.Hc) {
        p.gathered[row] = take ? static_cast<int32_t>(target_of(p.target, p.i32, i)) : -1;
        p.place[row] = take ? row : -1;
      }
    }
  }
  if (p.Hc) {
    const int64_t t = target_of(p.target, p.i32, blockIdx.x);
    const bool take = t >= 0 && t < p.V;
    const uint16_t *src = p.H + blockIdx.x * p.ldh;
    uint16_t *dst = p.Hc + blockIdx.x * p.ldc;
    for (int c = threadIdx.x * 8; c < p.D; c += 8192) {
      if (c + 8 <= p.D) {
        *reinterpret_cast<uint4 *>(dst + c) = take ? *reinterpret_cast<const uint4 *>(src + c) : make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (int e = c; e < p.D; ++e) dst[e] = take ? src[e] : uint16_t(0);
      }
    }
  }
  if (lane == 0) sums[warp] = make_float4(sum.x, sum.y, sum.z, 0.f);
  __syncthreads();
  if (warp > 0 && gridDim.x == 1) return;
  if (warp == 0) {
    sum = add_over_warp(make_float3(sums[lane].x, sums[lane].y, sums[lane].z));
    if (lane == 0 && gridDim.x > 1) {
      p.block_sums[blockIdx.x] = make_float4(sum.x, sum.y, sum.z, 0.f);
      __threadfence();
      last = atomicAdd(&p.sc->ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  if (gridDim.x > 1) {
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = make_float3(0.f, 0.f, 0.f);
    for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += 1024) {
      const float4 v = __ldcg(p.block_sums + b);
      sum = make_float3(sum.x + v.x, sum.y + v.y, fmaxf(sum.z, v.z));
    }
    sum = add_over_warp(sum);
    if (lane == 0) sums[warp] = make_float4(sum.x, sum.y, sum.z, 0.f);
    __syncthreads();
    if (warp > 0) return;
    sum = add_over_warp(make_float3(sums[lane].x, sums[lane].y, sums[lane].z));
  }
  if (lane == 0) {
    const float norm = p.mean ? sum.y : 1.f;
    if (p.total) *p.total = norm != 0.f ? sum.x / norm : 0.f;
    if (p.Hc) choose_split(p.split, p.T, p.sc);
    if (p.coef) {
      // dl is at most `big`: brought just below 2^14, clear of fp16's largest value
      // (65504) and of its subnormals for every p above 2^-28
      int e = 0;
      if (sum.z > 0.f) frexpf(sum.z, &e);
      e = max(-100, min(100, 14 - e));
      p.sc->dl_scale = ldexpf(1.f, e);
      p.sc->out_scale = norm != 0.f ? ldexpf(p.grad_scale / norm * p.c, -e) : 0.f;
    }
  }
}

struct ConvertParams {
  uint16_t *buf;             // [T][pitch]: kept distances in, dl out
  const float2 *stats;       // [slots][T]
  const float *at_target, *lse2;
  const float2 *coef;
  const int32_t *gathered;
  const XentScalars *sc;
  int64_t pitch;
  int32_t T, N, bn;          // N columns exist of the piece
  int32_t band, band_tiles;  // as in the product that kept them
  int32_t row_ctas;          // CTAs that share the rows of 512 columns
  float c2, c;               // logit_scale log2(e), logit_scale
};

// Kept distances to dl, in place: a warp per row of 512 columns, two times 16 bytes per
// lane, two rows ahead.  Bound by memory: 4 bytes and one exponential per logit (4096 x 32000 in 85 us alone,
// 6.1 TB/s).
constexpr int kConvertRows = 16;   // rows of a CTA (8 warps, 2 rows each)
constexpr int kConvertCols = 512;
__global__ void __launch_bounds__(256) xent_convert_kernel(const __grid_constant__ ConvertParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int rows = p.sc->rows;
  const int end = min(p.T, (rows + BK - 1) / BK * BK);  // zeros up to the next k-block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // last columns first: the product wrote them last, and what is left in L2 for
  // the next product is what that reads first
  const int across = gridDim.x / p.row_ctas, by = blockIdx.x / p.row_ctas, bx = blockIdx.x - by * p.row_ctas;
  const int c0 = (across - 1 - by) * kConvertCols + lane * 8;
  int64_t slot[2];
  bool there[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = c0 + 256 * h;
    slot[h] = int64_t(slot_of(c, p.N, p.band, p.band_tiles, p.bn)) * p.T;
    there[h] = c < (p.N + 255) / 256 * 256;
  }
  const float ds = p.sc->dl_scale;
  for (int first = bx * kConvertRows + warp; first < end; first += p.row_ctas * kConvertRows) {
    uint4 w[2][2];
    float top[2][2], lse2[2];
    float2 coef[2];
    int target[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = first + 8 * i;
      target[i] = -1;
      lse2[i] = 0.f;
      coef[i] = make_float2(0.f, 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[i][h] = make_uint4(0u, 0u, 0u, 0u);
        top[i][h] = 0.f;
      }
      if (r < rows) {
        const uint16_t *row = p.buf + r * p.pitch + c0;
        w[i][0] = *reinterpret_cast<const uint4 *>(row);
        if (there[1]) w[i][1] = *reinterpret_cast<const uint4 *>(row + 256);
        top[i][0] = p.stats[slot[0] + r].x;
        if (there[1]) top[i][1] = p.stats[slot[1] + r].x;
        lse2[i] = p.lse2[r];
        coef[i] = p.coef[r];
        target[i] = p.gathered[r];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = first + 8 * i;
      if (r >= end) continue;
      const bool live = target[i] >= 0;
      const float f = coef[i].x * ds;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!there[h]) continue;
        const int c = c0 + 256 * h, at = target[i] - c;
        const uint32_t u[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
        const float shift = (top[i][h] == -INFINITY ? 0.f : top[i][h]) - lse2[i];
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // the code in the low bits of a float of 2^23
          const float code = __uint_as_float(__byte_perm(u[e / 2], 0x4b000000u, e & 1 ? 0x7432 : 0x7410)) - 8388608.f;
          d[e] = ex2(fmaf(code, -1.f / (1 << kKeptBits), shift)) * f;
        }
        // the farthest code stands for every distance from there on: p is 0 (or NaN, like its row)
        const uint32_t most = __vmaxu2(__vmaxu2(u[0], u[1]), __vmaxu2(u[2], u[3]));
        if ((most & 0xffffu) == 0xffffu || most >> 16 == 0xffffu) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((u[e / 2] >> (16 * (e & 1)) & 0xffffu) == 0xffffu) d[e] *= 0.f;
        }
        if (live && at >= 0 && at < 8) {
          // the target's own logit is at hand in fp32: p - 1 loses nothing to the rounding of p
          const float v = ex2(p.at_target[r] * (p.c2 / p.c) - lse2[i]) * f - coef[i].y * ds;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e == at) d[e] = v;
        }
        if (!live || c + 8 > p.N) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!live || c + e >= p.N) d[e] = 0.f;
        }
        *reinterpret_cast<uint4 *>(p.buf + r * p.pitch + c) =
            make_uint4(pack16(true, d[0], d[1]), pack16(true, d[2], d[3]), pack16(true, d[4], d[5]),
                       pack16(true, d[6], d[7]));
      }
    }
  }
}

struct SpreadParams {
  const float *part;  // [slices][T][Dp]
  uint16_t *dH;
  const int32_t *place;
  const XentScalars *sc;
  int64_t lddh, Dp;
  int32_t T, D, bf16;
  SplitParams split;
  int32_t raster_group;
};

// Four columns of a row of dH per thread: its slices added in order; ignored rows are 0.
// kLanes threads share a quad's slices (every kLanes-th each, then the lanes in order),
// since a long chain of loads is what few rows with many slices would wait for.
template <int kLanes>
__global__ void __launch_bounds__(256) xent_spread_kernel(const __grid_constant__ SpreadParams p) {
  __shared__ float4 sums[kLanes > 1 ? 256 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const float scale = p.sc->out_scale;
  const int kbs = p.sc->kb_split, full = p.sc->full;
  const int m_blk = (p.sc->rows + p.split.m - 1) / p.split.m;
  constexpr int kQuads = 256 / kLanes;
  const int lane = threadIdx.x / kQuads;
  const int c = (blockIdx.x * kQuads + threadIdx.x % kQuads) * 4;
  for (int64_t i = blockIdx.y; i < p.T; i += gridDim.y) {
    const int r = p.place[i];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= 0 && c < p.D) {
      // the element's tile in the order of the product's tiles, and so its slices
      const int mb = r / p.split.m, group = mb / p.raster_group, first_m = group * p.raster_group;
      const int tile = first_m * p.split.n_blk + c / p.split.n * min(m_blk - first_m, p.raster_group) + mb - first_m;
      const int slices = tile < full ? 1 : (p.split.kb + kbs - 1) / kbs;
      const float *a = p.part + r * p.Dp + c;
#pragma unroll 8
      for (int s = lane; s < slices; s += kLanes) {
        const float4 f = *reinterpret_cast<const float4 *>(a + s * (p.T * p.Dp));
        v.x += f.x;
        v.y += f.y;
        v.z += f.z;
        v.w += f.w;
      }
    }
    if constexpr (kLanes > 1) {
      __syncthreads();  // the last row's sums have been read
      sums[threadIdx.x] = v;
      __syncthreads();
      if (lane > 0) continue;
#pragma unroll
      for (int l = 1; l < kLanes; ++l) {
        const float4 f = sums[threadIdx.x + l * kQuads];
        v = make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w);
      }
    }
    if (c >= p.D) continue;
    if (r >= 0) v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    const bool bf16 = p.bf16 != 0;
    const uint2 o = make_uint2(pack16(bf16, v.x, v.y), pack16(bf16, v.z, v.w));
    uint16_t *dst = p.dH + i * p.lddh + c;
    if (c + 4 <= p.D) {
      *reinterpret_cast<uint2 *>(dst) = o;
    } else {
      const uint32_t w[2] = {o.x, o.y};
      for (int e = 0; e < p.D - c; ++e) dst[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
    }
  }
}

// One product's tile shape and shared memory.
struct Product {
  int mode = X_STATS, cg = 1, bn = 128, stages = 2, boxes = 0;
  const void *fn = nullptr;
  uint32_t off_B = 0, off_out = 0, off_bar = 0;
};

cudaError_t launch(const void *fn, dim3 grid, int threads, int smem, int cluster, void *params, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  void *args[] = {params};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

struct Workspace {
  size_t scalars, index, place, gathered, gweight, at_target, lse2, coef, block_sums, stats, Hc, dl, part,
      bytes;
};

}  // namespace

struct gemm_epi_xent_plan {
  int64_t T = 0, V = 0, D = 0;
  ge_xent_desc d{};
  int sms = 0, smem = 0, pairs = 0;
  uint32_t *status = nullptr;
  Product stats, keep, dlogit, out, part;
  int64_t piece = 0;    // vocabulary columns of a piece, a multiple of 256
  int slices = 1;       // of dH's sum over a piece, at most
  bool pack_loss = true, pack_step = true;  // rows that take part are packed first
  int row_lanes = 32, finish_grid = 1;
  int64_t ldc = 0, Dp = 0;
  int64_t band = 0;     // columns of a CTA's band in the logits' product, 0: tiles
};

namespace {

// column ranges that leave a maximum and a sum
int slots_of(const gemm_epi_xent_plan *pl) {
  return static_cast<int>(ge::slots_of(pl->V, pl->band, pl->stats.bn));
}

Workspace workspace_of(const gemm_epi_xent_plan *pl, bool grads) {
  Workspace w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t T = static_cast<size_t>(pl->T);
  w.scalars = take(sizeof(XentScalars));
  w.index = take(4 * T);
  w.place = take(4 * T);
  w.gathered = take(4 * T);
  w.gweight = take(4 * T);
  w.at_target = take(4 * T);
  w.lse2 = take(4 * T);
  w.coef = take(8 * T);
  w.block_sums = take(16 * static_cast<size_t>(pl->finish_grid));
  w.stats = take(8 * T * static_cast<size_t>(slots_of(pl)));
  if (grads || pl->pack_loss) w.Hc = take(2 * T * static_cast<size_t>(pl->ldc));
  if (grads) {
    w.dl = take(2 * T * static_cast<size_t>(pl->piece));
    w.part = take(4 * T * static_cast<size_t>(pl->Dp) * static_cast<size_t>(pl->slices));
  }
  w.bytes = at + 256;  // to start on 256 bytes wherever the workspace does
  return w;
}

constexpr int kBarBytes = 1024, kAlignBytes = 1024;

int make_product(gemm_epi_xent_plan *pl, Product *pr, int mode, int cg, int boxes) {
  pr->mode = mode;
  pr->cg = cg;
  pr->bn = cg == 2 ? 256 : 128;
  pr->boxes = boxes;
  pr->fn = cg == 2 ? xent_kernel_cg2(mode) : xent_kernel_cg1(mode);
  const int stage = 32768;  // 128 rows of A and 128 of B, 64 of K, on either shape
  const int room = pl->smem - kBarBytes - kAlignBytes - 2 * boxes * static_cast<int>(kXentBox);
  pr->stages = std::min(kMaxStages, room / stage);
  if (pr->stages < 2) return GE_ERR_SMEM;
  pr->off_B = static_cast<uint32_t>(pr->stages * stage / 2);
  pr->off_out = static_cast<uint32_t>(pr->stages * stage);
  pr->off_bar = pr->off_out + 2u * static_cast<uint32_t>(boxes) * kXentBox;
  // all of an SM's shared memory: CTAs of two launches never share its TMEM
  if (cudaFuncSetAttribute(pr->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, pl->smem) != cudaSuccess)
    return GE_ERR_CUDA;
  return GE_OK;
}

int units_of(const gemm_epi_xent_plan *pl, const Product &pr) {
  int sms = pl->sms;
  if (pl->d.max_ctas) sms = std::min(sms, pl->d.max_ctas);
  return std::max(1, pr.cg == 2 ? std::min(pl->pairs, sms / 2) : sms);
}

int64_t tiles_of(const Product &pr, int64_t M, int64_t N) { return ceil_div(M, 128 * pr.cg) * ceil_div(N, pr.bn); }

int configure(gemm_epi_xent_plan *pl) {
  // Tiles: 256 x 256 on CTA pairs, or 128 x 128 on single CTAs where a batch fills no more
  // rows than that or the whole product is at most one tile for every SM, which
  // is then bound by its start and its end (256 x 8000 x 1024: a loss 17.0 us against
  // 18.9 on pairs, a step 54.5 against 59.7).
  const int sms = pl->d.max_ctas ? std::min(pl->d.max_ctas, pl->sms) : pl->sms;
  auto single = [&](int64_t M, int64_t N) { return ceil_div(M, 128) * ceil_div(N, 128) <= sms; };
  const int cg = sms < 2 || pl->T <= 128 || single(pl->T, pl->V) ? 1 : 2;
  // The gradients' products too, up to 10^10 operations (about 6 us of the GPU): 200 x 4000 x 512
  // in 36.7 us against 45.5, 1500 x 1000 x 2048 in 63.3 against 67.6.  And dW of up to 128 rows, which
  // is bound by its stores: 64 x 32000 x 2048 in 122 us against 129.
  const bool light = 2.0 * double(pl->T) * double(pl->V) * double(pl->D) <= 1e10;
  const int cg_out = sms < 2 || pl->T <= 128 || (light && single(pl->V, pl->D)) ? 1 : 2;
  const int cg_part = sms < 2 || pl->T <= 128 || (light && single(pl->T, pl->D)) ? 1 : 2;
  int st = make_product(pl, &pl->stats, X_STATS, cg, 0);
  if (st == GE_OK) st = make_product(pl, &pl->keep, X_KEEP, cg, 0);
  if (st == GE_OK) st = make_product(pl, &pl->dlogit, X_DLOGIT, cg, 0);
  if (st == GE_OK) st = make_product(pl, &pl->out, X_OUT, cg_out, 0);
  if (st == GE_OK) st = make_product(pl, &pl->part, X_PART, cg_part, kXentBoxes);
  if (st != GE_OK) return st;
  pl->pairs = pl->sms / 2;
  if (cudaFuncSetAttribute(xent_kernel_cg2(X_OUT), cudaFuncAttributeMaxDynamicSharedMemorySize, pl->smem) != cudaSuccess)
    return GE_ERR_CUDA;
  if (sms >= 2) {
    int clusters = 0;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kXentThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(pl->smem);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&clusters, xent_kernel_cg2(X_OUT), &cfg) == cudaSuccess && clusters > 0)
      pl->pairs = std::min(pl->pairs, clusters);
    cudaGetLastError();
  }
  // One tile of rows: its time is that of reading W, and every CTA is given as many of W's
  // rows as the next (to 32) where whole tiles would leave CTAs idle at the end (32000 rows:
  // 224 to a CTA instead of one or two tiles of 128).
  pl->band = cg == 1 && pl->T <= 128 ? band_of(pl->V, units_of(pl, pl->stats)) : 0;
  // Packing costs a launch (4 to 5 us) and saves the products of ignored rows: it is left
  // out where a batch fills one tile anyway and where the logits' product takes less than
  // about 20 us.  (A step without it needs a block of finish for every row.)
  const bool small = pl->T <= 128 || 2.0 * double(pl->T) * double(pl->V) * double(pl->D) < 3e10;
  pl->pack_loss = !small;
  pl->pack_step = !small || pl->T > 2 * pl->sms;
  pl->piece = piece_of(pl->T, pl->V, pl->d.buffer_bytes ? pl->d.buffer_bytes : int64_t(1) << 29);
  // dH: slices of its sum over a piece, decided on the device by the rows that
  // take part, within 64 MiB or what four waves of CTAs take of the tiles left over
  const int64_t tiles = tiles_of(pl->part, pl->T, pl->D);
  const int64_t kb = ceil_div(std::min(pl->piece, pl->V), BK);
  const int64_t fit = (int64_t(64) << 20) / (4 * pl->T * pl->Dp);
  const int64_t units = units_of(pl, pl->part), left = tiles % units;
  const int64_t want = left ? 4 * units / left : 1;
  pl->slices = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({std::max(fit, std::min<int64_t>(want, 8)), kb, 64})));
  // finish: a block of 1024 threads per row while that is at most two blocks to an SM, then up
  // to 32 rows to a block (37 rows of 858 ranges: 37 blocks 6 us, 2 blocks 11 us)
  pl->row_lanes = 1;
  while (pl->row_lanes < 32 && ceil_div(pl->T, pl->row_lanes) > 2 * int64_t(pl->sms)) pl->row_lanes *= 2;
  const int64_t fg = ceil_div(pl->T, pl->row_lanes);
  pl->finish_grid = static_cast<int>(fg);
  for (const Product *pr : {&pl->stats, &pl->part})
    if (tiles_of(*pr, pl->T, std::max(pl->V, pl->D)) * pl->slices > (int64_t(1) << 30)) return GE_ERR_SHAPE;
  return GE_OK;
}

// rows of a K-major A tile: all 128, or those of a batch that fills no tile
int64_t a_rows_of(const gemm_epi_xent_plan *pl, const Product &pr) {
  return pr.cg == 1 ? std::min<int64_t>(128, round_up(pl->T, 8)) : 128;
}

XentParams params_of(const gemm_epi_xent_plan *pl, const Product &pr, XentScalars *sc, int64_t M, int64_t N,
                     int64_t K) {
  XentParams p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  p.status = pl->status;
  p.timeout_ns = static_cast<uint64_t>(pl->d.timeout_ms ? pl->d.timeout_ms : 1000) * 1000000ull;
  p.sc = sc;
  p.rows = &sc->rows;
  p.all_rows = static_cast<int32_t>(pl->T);
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.num_n_blk = static_cast<int32_t>(ceil_div(N, pr.bn));
  const int64_t m_blk = ceil_div(M, 128 * pr.cg);
  p.raster_group = m_blk <= 16 ? 16 : 12;
  p.stages = pr.stages;
  p.debug_flags = pl->d.debug_flags;
  p.a_rows = static_cast<int32_t>(a_rows_of(pl, pr));
  p.bf16 = pl->d.ab == GE_BF16;
  p.off_B = pr.off_B;
  p.off_out = pr.off_out;
  p.off_bar = pr.off_bar;
  p.c = pl->d.logit_scale;
  p.c2 = pl->d.logit_scale * kLog2e;
  p.out_scale = &sc->out_scale;
  return p;
}

cudaError_t launch_product(const gemm_epi_xent_plan *pl, const Product &pr, XentParams &p, cudaStream_t s) {
  const int64_t tiles = p.band ? ceil_div(p.N, p.band) : tiles_of(pr, p.M, p.N) * (pr.mode == X_PART ? pl->slices : 1);
  const int units = static_cast<int>(std::min<int64_t>(units_of(pl, pr), tiles));
  // dW: a last wave that would leave half of the CTAs idle runs as half tiles
  const int64_t last = tiles % units_of(pl, pr);
  p.num_full = static_cast<int32_t>(last > 0 && 2 * last <= units_of(pl, pr) && tiles > last ? tiles - last : tiles);
  return launch(pr.fn, dim3(static_cast<unsigned>(units * pr.cg)), kXentThreads, pl->smem, pr.cg, &p, s);
}

int run(gemm_epi_xent_plan *pl, bool grads, const void *H, const void *W, const void *target, const float *weight,
        float grad_scale, float *loss, float *lse, float *total, void *dH, void *dW, void *workspace,
        size_t workspace_bytes, cudaStream_t s) {
  if (!pl) return GE_ERR_INVALID;
  if (!H || !W || !target) return GE_ERR_MISSING_ARG;
  if (grads && !dH && !dW) return GE_ERR_MISSING_ARG;
  for (const void *q : {H, W, target, static_cast<const void *>(weight), static_cast<const void *>(loss),
                        static_cast<const void *>(lse), static_cast<const void *>(total),
                        static_cast<const void *>(dH), static_cast<const void *>(dW)})
    if (!is_aligned16(q)) return GE_ERR_MISALIGNED;
  if (!std::isfinite(grad_scale)) return GE_ERR_INVALID;
  const Workspace at = workspace_of(pl, grads);
  if (!workspace || !is_aligned16(workspace) || workspace_bytes < at.bytes) return GE_ERR_WORKSPACE;
  // the buffers in it start on 256 bytes
  char *ws = reinterpret_cast<char *>(round_up(static_cast<int64_t>(reinterpret_cast<uintptr_t>(workspace)), 256));
  const int64_t T = pl->T, V = pl->V, D = pl->D;
  const int ab = pl->d.ab;
  XentScalars *sc = reinterpret_cast<XentScalars *>(ws + at.scalars);
  int32_t *index = reinterpret_cast<int32_t *>(ws + at.index);
  int32_t *place = reinterpret_cast<int32_t *>(ws + at.place);
  int32_t *gathered = reinterpret_cast<int32_t *>(ws + at.gathered);
  float *gweight = reinterpret_cast<float *>(ws + at.gweight);
  float *at_target = reinterpret_cast<float *>(ws + at.at_target);
  float *lse2 = reinterpret_cast<float *>(ws + at.lse2);
  float2 *coef = reinterpret_cast<float2 *>(ws + at.coef);
  float2 *stats = reinterpret_cast<float2 *>(ws + at.stats);
  void *Hc = ws + at.Hc;
  void *dl = ws + at.dl;
  float *part = reinterpret_cast<float *>(ws + at.part);
  const uint64_t piece = static_cast<uint64_t>(pl->piece);
  const bool pack = grads ? pl->pack_step : pl->pack_loss;
  const int i32 = pl->d.index == GE_INDEX_I32;
  const SplitParams split = {128 * pl->part.cg, pl->part.bn, static_cast<int32_t>(ceil_div(D, pl->part.bn)),
                             static_cast<int32_t>(ceil_div(std::min(pl->piece, V), BK)), units_of(pl, pl->part),
                             pl->slices};
  cudaError_t err = cudaSuccess;
  auto go = [&](cudaError_t e) { return (err = e) == cudaSuccess; };

  if (pack) {
    PackParams pp;
    std::memset(static_cast<void *>(&pp), 0, sizeof(pp));
    pp.target = target;
    pp.weight = weight;
    pp.H = static_cast<const uint16_t *>(H);
    pp.Hc = static_cast<uint16_t *>(Hc);
    pp.loss = loss;
    pp.lse = lse;
    pp.sc = sc;
    pp.index = index;
    pp.place = place;
    pp.gathered = gathered;
    pp.gweight = gweight;
    pp.V = V;
    pp.ldh = pl->d.ldh;
    pp.ldc = pl->ldc;
    pp.T = static_cast<int32_t>(T);
    pp.D = static_cast<int32_t>(D);
    pp.i32 = i32;
    const int ctas = static_cast<int>(std::min<int64_t>(ceil_div(T, 8), 2 * pl->sms));
    pp.rows_per_cta = static_cast<int32_t>(ceil_div(T, ctas));
    pp.split = split;
    if (!go(launch(reinterpret_cast<const void *>(xent_pack_kernel), ctas, kPackThreads, 0, 1, &pp, s)))
      return GE_ERR_CUDA;
  }

  const bool kept = grads && ab == GE_BF16;  // fp16: see kKeptBits
  const Product &first = kept ? pl->keep : pl->stats;
  XentParams sl = params_of(pl, first, sc, T, V, D);
  if (!encode_rows(&sl.tmA, ab, pack ? Hc : H, D, T, 1, pack ? pl->ldc : pl->d.ldh,
                   (pack ? pl->ldc : pl->d.ldh) * T, BK, sl.a_rows) ||
      !encode_rows(&sl.tmH, ab, H, D, T, 1, pl->d.ldh, pl->d.ldh * T, BK, sl.a_rows) ||
      !encode_rows(&sl.tmB, ab, W, D, V, 1, pl->d.ldw, pl->d.ldw * V, BK, 128) ||
      (pl->band && !encode_rows(&sl.tmB32, ab, W, D, V, 1, pl->d.ldw, pl->d.ldw * V, BK, 32)))
    return GE_ERR_CUDA;
  sl.band = static_cast<int32_t>(pl->band);
  sl.band_tiles = static_cast<int32_t>(pl->band ? ceil_div(pl->band, first.bn) : 0);
  if (!pack) sl.rows = nullptr;
  sl.target = pack ? static_cast<const void *>(gathered) : target;
  sl.target_i64 = !pack && !i32;
  sl.stats = stats;
  sl.at_target = at_target;
  if (kept) {
    sl.keep_cols = static_cast<int32_t>(std::min<int64_t>(pl->piece, round_up(V, 256)));
    sl.out = static_cast<uint16_t *>(dl);
    sl.ld_out = pl->piece;
  }
  if (!go(launch_product(pl, first, sl, s))) return GE_ERR_CUDA;

  FinishParams fp;
  std::memset(static_cast<void *>(&fp), 0, sizeof(fp));
  fp.stats = stats;
  fp.at_target = at_target;
  fp.index = pack ? index : nullptr;
  fp.gweight = gweight;
  fp.target = target;
  fp.weight = weight;
  fp.loss = loss;
  fp.lse = lse;
  fp.total = total;
  fp.lse2 = lse2;
  fp.coef = grads ? coef : nullptr;
  fp.block_sums = reinterpret_cast<float4 *>(ws + at.block_sums);
  fp.sc = sc;
  fp.V = V;
  fp.T = static_cast<int32_t>(T);
  fp.i32 = i32;
  fp.slots = slots_of(pl);
  fp.row_lanes = pl->row_lanes;
  if (grads && !pack) {
    fp.H = static_cast<const uint16_t *>(H);
    fp.Hc = static_cast<uint16_t *>(Hc);
    fp.gathered = gathered;
    fp.place = place;
    fp.ldh = pl->d.ldh;
    fp.ldc = pl->ldc;
    fp.split = split;
  }
  fp.D = static_cast<int32_t>(D);
  fp.mean = pl->d.reduction == GE_XENT_MEAN;
  fp.z = pl->d.z_loss;
  fp.grad_scale = grad_scale;
  fp.c = pl->d.logit_scale;
  if (!go(launch(reinterpret_cast<const void *>(xent_finish_kernel), pl->finish_grid, 1024, 0, 1, &fp, s)))
    return GE_ERR_CUDA;
  if (!grads) return GE_OK;

  for (int64_t v0 = 0; v0 < V; v0 += pl->piece) {
    const int64_t n = std::min(pl->piece, V - v0);
    if (kept && v0 == 0) {
      ConvertParams cp;
      std::memset(static_cast<void *>(&cp), 0, sizeof(cp));
      cp.buf = static_cast<uint16_t *>(dl);
      cp.stats = stats;
      cp.at_target = at_target;
      cp.lse2 = lse2;
      cp.coef = coef;
      cp.gathered = gathered;
      cp.sc = sc;
      cp.pitch = pl->piece;
      cp.T = static_cast<int32_t>(T);
      cp.N = static_cast<int32_t>(n);
      cp.bn = first.bn;
      cp.band = sl.band;
      cp.band_tiles = sl.band_tiles;
      cp.c2 = sl.c2;
      cp.c = sl.c;
      const int64_t cols = ceil_div(n, kConvertCols);
      cp.row_ctas = static_cast<int32_t>(
          std::max<int64_t>(1, std::min<int64_t>(ceil_div(T, kConvertRows), ceil_div(16 * pl->sms, cols))));
      const dim3 grid(static_cast<unsigned>(cols * cp.row_ctas));
      if (!go(launch(reinterpret_cast<const void *>(xent_convert_kernel), grid, 256, 0, 1, &cp, s)))
        return GE_ERR_CUDA;
    } else {
      XentParams q = params_of(pl, pl->dlogit, sc, T, n, D);
      q.tmA = sl.tmA;
      q.tmH = sl.tmH;
      q.b_row0 = static_cast<int32_t>(v0);
      q.target = gathered;
      q.lse2 = lse2;
      q.coef = coef;
      q.out = static_cast<uint16_t *>(dl);
      q.ld_out = pl->piece;
      q.tmB = sl.tmB;
      if (!go(launch_product(pl, pl->dlogit, q, s))) return GE_ERR_CUDA;
    }
    if (dW) {
      XentParams o = params_of(pl, pl->out, sc, n, D, T);
      if (!pack) o.all_rows = static_cast<int32_t>(T) + 1;  // rows that take no part are zeros in Hc alone
      o.out = static_cast<uint16_t *>(dW);
      o.ld_out = pl->d.lddw;
      o.out32 = pl->d.lddw % 16 == 0 && reinterpret_cast<uintptr_t>(dW) % 32 == 0;
      o.b_row0 = static_cast<int32_t>(v0);
      if (!encode_rows(&o.tmA, ab, dl, piece, T, 1, piece, piece * T, 64, BK) ||
          !encode_rows(&o.tmB, ab, Hc, D, T, 1, pl->ldc, pl->ldc * T, 64, BK) ||
          !encode_rows(&o.tmH, ab, H, D, T, 1, pl->d.ldh, pl->d.ldh * T, 64, BK) ||
          !go(launch_product(pl, pl->out, o, s)))
        return GE_ERR_CUDA;
    }
    if (dH) {
      XentParams o = params_of(pl, pl->part, sc, T, D, n);
      o.b_row0 = static_cast<int32_t>(v0);
      o.accumulate = v0 > 0;
      if (!encode_rows(&o.tmA, ab, dl, piece, T, 1, piece, piece * T, BK, o.a_rows) ||
          !encode_rows(&o.tmB, ab, W, D, V, 1, pl->d.ldw, pl->d.ldw * V, 64, BK) ||
          !encode_rows(&o.tmOut, GE_F32, part, pl->Dp, T, pl->slices, pl->Dp, pl->Dp * T, 32, 128) ||
          !go(launch_product(pl, pl->part, o, s)))
        return GE_ERR_CUDA;
    }
  }
  if (dH) {
    SpreadParams dp{part, static_cast<uint16_t *>(dH), place, sc, pl->d.lddh, pl->Dp, static_cast<int32_t>(T),
                    static_cast<int32_t>(D), ab == GE_BF16, split, params_of(pl, pl->part, sc, T, D, 1).raster_group};
    const bool shared = pl->slices > 8;
    const int64_t across = ceil_div(D, shared ? 128 : 1024);
    const dim3 grid(static_cast<unsigned>(across),
                    static_cast<unsigned>(std::min<int64_t>(T, std::max<int64_t>(1, pl->sms * 16 / across))));
    const void *fn = shared ? reinterpret_cast<const void *>(xent_spread_kernel<8>)
                            : reinterpret_cast<const void *>(xent_spread_kernel<1>);
    if (!go(launch(fn, grid, 256, 0, 1, &dp, s))) return GE_ERR_CUDA;
  }
  return GE_OK;
}

}  // namespace

extern "C" {

int gemm_epi_xent_plan_create(gemm_epi_xent_plan **plan, int64_t T, int64_t V, int64_t D, const ge_xent_desc *desc) {
  if (!plan) return GE_ERR_INVALID;
  *plan = nullptr;
  if (!desc) return GE_ERR_INVALID;
  if (desc->ab != GE_F16 && desc->ab != GE_BF16) return GE_ERR_UNSUPPORTED;
  if (desc->index != GE_INDEX_I64 && desc->index != GE_INDEX_I32) return GE_ERR_UNSUPPORTED;
  if ((desc->reduction != GE_XENT_SUM && desc->reduction != GE_XENT_MEAN) || desc->timeout_ms < 0 ||
      desc->max_ctas < 0 || (desc->debug_flags & ~GE_DEBUG_SKIP_FIRST_LOAD) != 0 || desc->buffer_bytes < 0 || !std::isfinite(desc->logit_scale) ||
      !std::isfinite(desc->z_loss))
    return GE_ERR_INVALID;
  const int64_t most = (int64_t(1) << 31) - 1;
  if (T <= 0 || V <= 0 || D <= 0 || T > most || V > most - 256 || D > most) return GE_ERR_SHAPE;
  ge_xent_desc d = *desc;
  if (d.logit_scale == 0.f) d.logit_scale = 1.f;
  for (int64_t *ld : {&d.ldh, &d.ldw, &d.lddh, &d.lddw}) {
    if (*ld == 0) *ld = D;
    if (*ld < D || *ld > most) return GE_ERR_SHAPE;
    if (*ld % 8 != 0) return GE_ERR_MISALIGNED;
  }
  gemm_epi_xent_plan *pl = new (std::nothrow) gemm_epi_xent_plan();
  if (!pl) return GE_ERR_INVALID;
  pl->T = T;
  pl->V = V;
  pl->D = D;
  pl->d = d;
  pl->ldc = round_up(D, 8);
  pl->Dp = round_up(D, 8);
  int dev = 0;
  int st = current_device(&dev, &pl->sms, &pl->smem);
  if (st == GE_OK) {
    pl->status = status_block();
    if (!pl->status) st = GE_ERR_CUDA;
  }
  if (st == GE_OK) st = configure(pl);
  if (st != GE_OK) {
    cudaGetLastError();
    delete pl;
    return st;
  }
  *plan = pl;
  return GE_OK;
}

void gemm_epi_xent_plan_destroy(gemm_epi_xent_plan *plan) { delete plan; }

size_t gemm_epi_xent_workspace_bytes(const gemm_epi_xent_plan *plan, int grads) {
  return plan ? workspace_of(plan, grads != 0).bytes : 0;
}

int gemm_epi_xent_loss(gemm_epi_xent_plan *plan, const void *H, const void *W, const void *target,
                       const float *weight, float *loss, float *lse, float *total, void *workspace,
                       size_t workspace_bytes, void *stream) {
  return run(plan, false, H, W, target, weight, 1.f, loss, lse, total, nullptr, nullptr, workspace, workspace_bytes,
             static_cast<cudaStream_t>(stream));
}

int gemm_epi_xent_step(gemm_epi_xent_plan *plan, const void *H, const void *W, const void *target,
                       const float *weight, float grad_scale, float *loss, float *lse, float *total, void *dH,
                       void *dW, void *workspace, size_t workspace_bytes, void *stream) {
  return run(plan, true, H, W, target, weight, grad_scale, loss, lse, total, dH, dW, workspace, workspace_bytes,
             static_cast<cudaStream_t>(stream));
}

}  // extern "C"
