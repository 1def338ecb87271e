// xent.cu -- the vocabulary loss and its gradients (gemm_epi_xent_*): plan,
// launches, and the small kernels around the products of xent_kernel.cuh.
//
//   scan     one CTA: which rows take part (their target exists), their order,
//            targets and weights; ignored rows get loss and lse 0
//   gather   their hidden states, packed; up to a k-block of zero rows after
//   X_STATS  logits -> per row and column range: maximum, sum, target's logit
//   finish   joins the ranges: lse, loss, total; what the gradients need per row
//   per piece of the vocabulary:
//     X_DLOGIT  dl of the piece (16 bits)
//     X_OUT     dW rows of the piece = dl^T @ H
//     X_PART    dH += dl @ W, fp32
//   spread   dH slices added in order, rounded, back to the rows' places
//
// Few kernels know how many rows take part; all read it from device memory.
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

using namespace ge;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994531;

// Device scalars of a run, at the start of the workspace.
struct Scalars {
  int32_t rows;       // rows that take part
  int32_t ticket;     // finish blocks done
  double weights;     // sum of their weights
  float out_scale;    // multiplies dl @ W and dl^T @ H
  float dl_scale;     // power of two in dl
};

struct ScanParams {
  const void *target;
  const float *weight;
  float *loss, *lse;
  Scalars *sc;
  int32_t *index, *place, *gathered;  // row of the r-th taken, its inverse (-1: ignored), targets
  float *gweight;
  int64_t V;
  int32_t T, i32;
};

__device__ __forceinline__ int64_t target_of(const void *t, int i32, int64_t i) {
  return i32 ? static_cast<const int32_t *>(t)[i] : static_cast<const int64_t *>(t)[i];
}

// Rows in order: a ballot within each warp, a scan over the CTA's warps, and a
// running count from chunk to chunk of 1024 rows.
__global__ void __launch_bounds__(1024) xent_scan_kernel(const __grid_constant__ ScanParams p) {
  __shared__ int counts[32];
  __shared__ double sums[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  double w_sum = 0.0;
  for (int64_t first = 0; first < p.T; first += 1024) {
    const int64_t i = first + threadIdx.x;
    const int64_t t = i < p.T ? target_of(p.target, p.i32, i) : -1;
    const bool take = t >= 0 && t < p.V;
    const unsigned vote = __ballot_sync(0xffffffffu, take);
    if (lane == 0) counts[warp] = __popc(vote);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      before += w < warp ? counts[w] : 0;
      all += counts[w];
    }
    __syncthreads();
    if (take) {
      const int r = base + before + __popc(vote & ((1u << lane) - 1u));
      const float w = p.weight ? p.weight[i] : 1.f;
      p.index[r] = static_cast<int32_t>(i);
      p.gathered[r] = static_cast<int32_t>(t);
      p.gweight[r] = w;
      p.place[i] = r;
      w_sum += w;
    } else if (i < p.T) {
      p.place[i] = -1;
      if (p.loss) p.loss[i] = 0.f;
      if (p.lse) p.lse[i] = 0.f;
    }
    base += all;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) w_sum += __shfl_xor_sync(0xffffffffu, w_sum, s);
  if (lane == 0) sums[warp] = w_sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < 32; ++w) s += sums[w];
    p.sc->rows = base;
    p.sc->ticket = 0;
    p.sc->weights = s;
  }
}

struct GatherParams {
  const uint16_t *H;
  uint16_t *Hc;
  const int32_t *index;
  const Scalars *sc;
  int64_t ldh, ldc;
  int32_t T, D;
};

// A warp per row, 16 bytes per lane.
__global__ void __launch_bounds__(256) xent_gather_kernel(const __grid_constant__ GatherParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int rows = p.sc->rows;
  const int end = min(p.T, (rows + BK - 1) / BK * BK);
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < end; r += gridDim.x * 8) {
    const uint16_t *src = r < rows ? p.H + int64_t(p.index[r]) * p.ldh : nullptr;
    uint16_t *dst = p.Hc + r * p.ldc;
    for (int c = lane * 8; c < p.D; c += 256) {
      if (c + 8 <= p.D) {
        *reinterpret_cast<uint4 *>(dst + c) =
            src ? *reinterpret_cast<const uint4 *>(src + c) : make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (int i = c; i < p.D; ++i) dst[i] = src ? src[i] : uint16_t(0);
      }
    }
  }
}

struct FinishParams {
  const float2 *stats;       // [slots][T]
  const float *at_target;
  const int32_t *index;
  const float *gweight;
  float *loss, *lse, *total;
  float *lse2;
  float2 *coef;
  double *block_sum;         // per block
  float *block_top;
  Scalars *sc;
  int32_t T, slots, row_lanes;  // row_lanes rows per block of 1024 threads
  int32_t mean;
  float z, grad_scale, c;
};

// row_lanes consecutive rows per block; the other threads share each row's
// column ranges: maxima first, then the sums brought to their maximum.  The
// last block to finish adds the blocks' sums in order.
__global__ void __launch_bounds__(1024) xent_finish_kernel(const __grid_constant__ FinishParams p) {
  __shared__ float fbuf[1024];
  __shared__ double dbuf[32];
  __shared__ bool last;
  griddep_wait();
  griddep_launch_dependents();
  const int rows = p.sc->rows;
  const int per = p.row_lanes, lanes = 1024 / per;
  const int x = threadIdx.x % per, y = threadIdx.x / per;
  const int r = blockIdx.x * per + x;
  const bool on = r < rows;
  float top = -INFINITY;
  if (on)
#pragma unroll 8
    for (int s = y; s < p.slots; s += lanes) top = fmaxf(top, p.stats[int64_t(s) * p.T + r].x);
  fbuf[threadIdx.x] = top;
  __syncthreads();
  for (int h = lanes / 2; h > 0; h >>= 1) {
    if (y < h) fbuf[threadIdx.x] = fmaxf(fbuf[threadIdx.x], fbuf[threadIdx.x + h * per]);
    __syncthreads();
  }
  top = fbuf[x];
  __syncthreads();
  const float off = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  if (on)
#pragma unroll 8
    for (int s = y; s < p.slots; s += lanes) {
      const float2 v = p.stats[int64_t(s) * p.T + r];
      sum += v.y * exp2f(v.x - off);
    }
  fbuf[threadIdx.x] = sum;
  __syncthreads();
  for (int h = lanes / 2; h > 0; h >>= 1) {
    if (y < h) fbuf[threadIdx.x] += fbuf[threadIdx.x + h * per];
    __syncthreads();
  }
  double loss = 0.0;
  float big = 0.f;
  if (y == 0 && on) {
    sum = fbuf[x];
    const double l2 = double(off) + log2(double(sum));
    const double lse = l2 * kLn2;
    const float w = p.gweight[r];
    const double at = p.at_target[r];
    loss = double(w) * (lse - at + double(p.z) * lse * lse);
    const int i = p.index[r];
    if (p.loss) p.loss[i] = static_cast<float>(loss);
    if (p.lse) p.lse[i] = static_cast<float>(lse);
    if (p.coef) {
      const float zf = static_cast<float>(1.0 + 2.0 * double(p.z) * lse);
      p.lse2[r] = static_cast<float>(l2);
      p.coef[r] = make_float2(w * zf, w);  // scaled by the last block's choice in xent_scale_kernel
      const float b = fabsf(w) * fmaxf(1.f, fabsf(zf));
      big = isfinite(b) ? b : 0.f;
    }
  }
  // rows of the block live in its first `per` (at most 32) threads
  if (threadIdx.x < 32) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      loss += __shfl_xor_sync(0xffffffffu, loss, s);
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
    }
    if (threadIdx.x == 0) {
      p.block_sum[blockIdx.x] = loss;
      p.block_top[blockIdx.x] = big;
      __threadfence();
      last = atomicAdd(&p.sc->ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // each thread adds every 1024th block, then the threads' sums are added in order
  double total = 0.0;
  big = 0.f;
  for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += 1024) {
    total += __ldcg(p.block_sum + b);
    big = fmaxf(big, __ldcg(p.block_top + b));
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, s);
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
  }
  if ((threadIdx.x & 31) == 0) {
    dbuf[threadIdx.x >> 5] = total;
    fbuf[threadIdx.x >> 5] = big;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    total = 0.0;
    big = 0.f;
    for (int w = 0; w < 32; ++w) {
      total += dbuf[w];
      big = fmaxf(big, fbuf[w]);
    }
    const double norm = p.mean ? p.sc->weights : 1.0;
    if (p.total) *p.total = norm != 0.0 ? static_cast<float>(total / norm) : 0.f;
    // dl is at most `big`: brought just below 2^14, clear of fp16's largest value
    // (65504) and of its subnormals for every p above 2^-28
    int e = 0;
    if (big > 0.f) frexpf(big, &e);
    e = max(-100, min(100, 14 - e));
    p.sc->dl_scale = ldexpf(1.f, e);
    p.sc->out_scale = norm != 0.0 ? static_cast<float>(ldexp(double(p.grad_scale) * double(p.c) / norm, -e)) : 0.f;
  }
}

// coef *= dl_scale
struct ScaleParams {
  float2 *coef;
  const Scalars *sc;
};
__global__ void __launch_bounds__(256) xent_scale_kernel(const __grid_constant__ ScaleParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const float s = p.sc->dl_scale;
  for (int r = blockIdx.x * 256 + threadIdx.x; r < p.sc->rows; r += gridDim.x * 256) {
    const float2 v = p.coef[r];
    p.coef[r] = make_float2(v.x * s, v.y * s);
  }
}

struct SpreadParams {
  const float *part;  // [slices][T][Dp]
  uint16_t *dH;
  const int32_t *place;
  const Scalars *sc;
  int64_t lddh, Dp;
  int32_t T, D, slices, bf16;
};

// A warp per row of dH: its slices added in order; ignored rows are 0.
__global__ void __launch_bounds__(256) xent_spread_kernel(const __grid_constant__ SpreadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const float scale = p.sc->out_scale;
  const int chunks = (p.D + 7) / 8;
  const int64_t units = int64_t(p.T) * chunks;
  for (int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x; u < units; u += int64_t(gridDim.x) * 256) {
    const int64_t i = u / chunks;
    const int c = static_cast<int>(u - i * chunks) * 8;
    const int r = p.place[i];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (r >= 0) {
      for (int s = 0; s < p.slices; ++s) {
        const float4 *a = reinterpret_cast<const float4 *>(p.part + (int64_t(s) * p.T + r) * p.Dp + c);
        const float4 lo = a[0], hi = a[1];
        v[0] += lo.x;
        v[1] += lo.y;
        v[2] += lo.z;
        v[3] += lo.w;
        v[4] += hi.x;
        v[5] += hi.y;
        v[6] += hi.z;
        v[7] += hi.w;
      }
    }
    union { uint16_t e[8]; uint4 w; } o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = r >= 0 ? v[e] * scale : 0.f;
      o.e[e] = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
    }
    uint16_t *dst = p.dH + i * p.lddh + c;
    if (c + 8 <= p.D) {
      *reinterpret_cast<uint4 *>(dst) = o.w;
    } else {
      for (int e = 0; e < p.D - c; ++e) dst[e] = o.e[e];
    }
  }
}

// One product's tile shape and shared memory.
struct Product {
  int mode = X_STATS, cg = 1, bn = 128, stages = 2, boxes = 0;
  const void *fn = nullptr;
  uint32_t off_B = 0, off_out = 0, off_bar = 0;
};

cudaError_t launch(const void *fn, int grid, int threads, int smem, int cluster, void *params, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
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
  size_t scalars, index, place, gathered, gweight, at_target, lse2, coef, block_sum, block_top, stats, Hc, dl, part,
      bytes;
};

}  // namespace

struct gemm_epi_xent_plan {
  int64_t T = 0, V = 0, D = 0;
  ge_xent_desc d{};
  int sms = 0, smem = 0, pairs = 0;
  uint32_t *status = nullptr;
  Product stats, dlogit, out, part;
  int64_t piece = 0;    // vocabulary columns of a piece, a multiple of 256
  int slices = 1, kb_split = 1;
  int row_lanes = 32, finish_grid = 1;
  int64_t ldc = 0, Dp = 0;
};

namespace {

int slots_of(const gemm_epi_xent_plan *pl) { return static_cast<int>(2 * ceil_div(pl->V, pl->stats.bn)); }

Workspace workspace_of(const gemm_epi_xent_plan *pl, bool grads) {
  Workspace w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t T = static_cast<size_t>(pl->T);
  w.scalars = take(sizeof(Scalars));
  w.index = take(4 * T);
  w.place = take(4 * T);
  w.gathered = take(4 * T);
  w.gweight = take(4 * T);
  w.at_target = take(4 * T);
  w.lse2 = take(4 * T);
  w.coef = take(8 * T);
  w.block_sum = take(8 * static_cast<size_t>(pl->finish_grid));
  w.block_top = take(4 * static_cast<size_t>(pl->finish_grid));
  w.stats = take(8 * T * static_cast<size_t>(slots_of(pl)));
  w.Hc = take(2 * T * static_cast<size_t>(pl->ldc));
  if (grads) {
    w.dl = take(2 * T * static_cast<size_t>(pl->piece));
    w.part = take(4 * T * static_cast<size_t>(pl->Dp) * static_cast<size_t>(pl->slices));
  }
  w.bytes = at;
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
  // A batch of at most 128 rows fills one 128-row tile; longer ones use CTA pairs.
  const int cg = pl->T <= 128 || (pl->d.max_ctas && pl->d.max_ctas < 2) ? 1 : 2;
  const int cg_out = pl->d.max_ctas && pl->d.max_ctas < 2 ? 1 : 2;
  int st = make_product(pl, &pl->stats, X_STATS, cg, 0);
  if (st == GE_OK) st = make_product(pl, &pl->dlogit, X_DLOGIT, cg, 2);
  if (st == GE_OK) st = make_product(pl, &pl->out, X_OUT, cg_out, 2);
  if (st == GE_OK) st = make_product(pl, &pl->part, X_PART, cg, 2);
  if (st != GE_OK) return st;
  pl->pairs = pl->sms / 2;
  if (cg_out == 2) {
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
    if (cudaOccupancyMaxActiveClusters(&clusters, pl->out.fn, &cfg) == cudaSuccess && clusters > 0)
      pl->pairs = std::min(pl->pairs, clusters);
    cudaGetLastError();
  }
  // pieces of the vocabulary: as wide as the buffer allows, equal, whole tiles
  const int64_t bound = pl->d.buffer_bytes ? pl->d.buffer_bytes : int64_t(1) << 30;
  const int64_t widest = std::max<int64_t>(256, bound / (2 * pl->T) / 256 * 256);
  const int64_t pieces = ceil_div(pl->V, widest);
  pl->piece = round_up(ceil_div(pl->V, pieces), 256);
  // dH: K (the piece) in as many slices as leave the fewest idle CTAs
  const int64_t tiles = tiles_of(pl->part, pl->T, pl->D);
  const int64_t kb = ceil_div(std::min(pl->piece, pl->V), BK);
  const int units = units_of(pl, pl->part);
  double best = 0;
  for (int64_t s = 1; s <= std::min<int64_t>(kb, 64); ++s) {
    const int64_t kbs = ceil_div(kb, s);
    if (ceil_div(kb, kbs) != s) continue;
    // in k-blocks of a tile (0.27 us each): waves of tiles, each its k-blocks and about
    // six k-blocks' time of set-up and stores, and each slice's way to memory and back
    const double cost = double(ceil_div(tiles * s, units)) * double(kbs + 6) +
                        double(s) * double(pl->T) * double(pl->D) * 8.0 / (6.5e6 * 0.27);
    if (s == 1 || cost < best * 0.97) {
      best = cost;
      pl->slices = static_cast<int>(s);
      pl->kb_split = static_cast<int>(kbs);
    }
  }
  // finish: few rows are shared by more threads each
  pl->row_lanes = 32;
  while (pl->row_lanes > 1 && pl->row_lanes / 2 >= pl->T) pl->row_lanes /= 2;
  const int64_t fg = ceil_div(pl->T, pl->row_lanes);
  pl->finish_grid = static_cast<int>(fg);
  for (const Product *pr : {&pl->stats, &pl->part})
    if (tiles_of(*pr, pl->T, std::max(pl->V, pl->D)) * 64 > (int64_t(1) << 30)) return GE_ERR_SHAPE;
  return GE_OK;
}

XentParams params_of(const gemm_epi_xent_plan *pl, const Product &pr, const Scalars *sc, int64_t M, int64_t N,
                     int64_t K) {
  XentParams p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  p.status = pl->status;
  p.timeout_ns = static_cast<uint64_t>(pl->d.timeout_ms ? pl->d.timeout_ms : 1000) * 1000000ull;
  p.rows = &sc->rows;
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.num_n_blk = static_cast<int32_t>(ceil_div(N, pr.bn));
  const int64_t m_blk = ceil_div(M, 128 * pr.cg);
  p.raster_group = m_blk <= 16 ? 16 : 12;
  p.splits = 1;
  p.kb_split = static_cast<int32_t>(ceil_div(K, BK));
  p.stages = pr.stages;
  p.boxes = pr.boxes;
  p.bf16 = pl->d.ab == GE_BF16;
  p.off_B = pr.off_B;
  p.off_out = pr.off_out;
  p.off_bar = pr.off_bar;
  p.c = pl->d.logit_scale;
  p.c2 = pl->d.logit_scale * kLog2e;
  p.out_scale = &sc->out_scale;
  return p;
}

cudaError_t launch_product(const gemm_epi_xent_plan *pl, const Product &pr, XentParams &p, int64_t splits,
                           cudaStream_t s) {
  const int64_t tiles = tiles_of(pr, p.M, p.N) * splits;
  const int units = static_cast<int>(std::min<int64_t>(units_of(pl, pr), tiles));
  return launch(pr.fn, units * pr.cg, kXentThreads, pl->smem, pr.cg, &p, s);
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
  char *ws = static_cast<char *>(workspace);
  const int64_t T = pl->T, V = pl->V, D = pl->D;
  const int ab = pl->d.ab;
  Scalars *sc = reinterpret_cast<Scalars *>(ws + at.scalars);
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
  const int spread_grid = pl->sms * 8;
  bool ok = true;
  auto go = [&](cudaError_t e) { ok = ok && e == cudaSuccess; };

  ScanParams sp{target, weight, loss, lse, sc, index, place, gathered, gweight, V, static_cast<int32_t>(T),
                pl->d.index == GE_INDEX_I32};
  go(launch(reinterpret_cast<const void *>(xent_scan_kernel), 1, 1024, 0, 1, &sp, s));
  GatherParams gp{static_cast<const uint16_t *>(H), static_cast<uint16_t *>(Hc), index, sc, pl->d.ldh, pl->ldc,
                  static_cast<int32_t>(T), static_cast<int32_t>(D)};
  go(launch(reinterpret_cast<const void *>(xent_gather_kernel),
            static_cast<int>(std::min<int64_t>(ceil_div(T, 8), spread_grid)), 256, 0, 1, &gp, s));

  XentParams sl = params_of(pl, pl->stats, sc, T, V, D);
  ok = ok && encode_rows(&sl.tmA, ab, Hc, D, T, 1, pl->ldc, pl->ldc * T, BK, 128);
  ok = ok && encode_rows(&sl.tmB, ab, W, D, V, 1, pl->d.ldw, pl->d.ldw * V, BK, 128);
  if (!ok) return GE_ERR_CUDA;
  sl.target = gathered;
  sl.stats = stats;
  sl.at_target = at_target;
  go(launch_product(pl, pl->stats, sl, 1, s));

  FinishParams fp;
  std::memset(static_cast<void *>(&fp), 0, sizeof(fp));
  fp.stats = stats;
  fp.at_target = at_target;
  fp.index = index;
  fp.gweight = gweight;
  fp.loss = loss;
  fp.lse = lse;
  fp.total = total;
  fp.lse2 = lse2;
  fp.coef = grads ? coef : nullptr;
  fp.block_sum = reinterpret_cast<double *>(ws + at.block_sum);
  fp.block_top = reinterpret_cast<float *>(ws + at.block_top);
  fp.sc = sc;
  fp.T = static_cast<int32_t>(T);
  fp.slots = slots_of(pl);
  fp.row_lanes = pl->row_lanes;
  fp.mean = pl->d.reduction == GE_XENT_MEAN;
  fp.z = pl->d.z_loss;
  fp.grad_scale = grad_scale;
  fp.c = pl->d.logit_scale;
  go(launch(reinterpret_cast<const void *>(xent_finish_kernel), pl->finish_grid, 1024, 0, 1, &fp, s));
  if (!grads) return ok ? GE_OK : GE_ERR_CUDA;

  ScaleParams cp{coef, sc};
  go(launch(reinterpret_cast<const void *>(xent_scale_kernel),
            static_cast<int>(std::min<int64_t>(ceil_div(T, 256), pl->sms)), 256, 0, 1, &cp, s));
  const uint64_t piece = static_cast<uint64_t>(pl->piece);
  for (int64_t v0 = 0; v0 < V; v0 += pl->piece) {
    const int64_t n = std::min(pl->piece, V - v0);
    XentParams q = params_of(pl, pl->dlogit, sc, T, n, D);
    q.tmA = sl.tmA;
    q.tmB = sl.tmB;
    ok = ok && encode_rows(&q.tmOut, ab, dl, piece, T, 1, piece, piece * T, 64, 128);
    q.b_row0 = static_cast<int32_t>(v0);
    q.target = gathered;
    q.lse2 = lse2;
    q.coef = coef;
    if (!ok) return GE_ERR_CUDA;
    go(launch_product(pl, pl->dlogit, q, 1, s));
    if (dW) {
      XentParams o = params_of(pl, pl->out, sc, n, D, T);
      ok = ok && encode_rows(&o.tmA, ab, dl, piece, T, 1, piece, piece * T, 64, BK);
      ok = ok && encode_rows(&o.tmB, ab, Hc, D, T, 1, pl->ldc, pl->ldc * T, 64, BK);
      o.tma_cols = static_cast<int32_t>(D / 8 * 8);
      o.out = static_cast<uint16_t *>(dW);
      o.ld_out = pl->d.lddw;
      if (o.tma_cols)
        ok = ok && encode_rows(&o.tmOut, ab, dW, o.tma_cols, V, 1, pl->d.lddw, pl->d.lddw * V, 64, 128);
      o.b_row0 = static_cast<int32_t>(v0);
      if (!ok) return GE_ERR_CUDA;
      go(launch_product(pl, pl->out, o, 1, s));
    }
    if (dH) {
      XentParams o = params_of(pl, pl->part, sc, T, D, n);
      ok = ok && encode_rows(&o.tmA, ab, dl, piece, T, 1, piece, piece * T, BK, 128);
      ok = ok && encode_rows(&o.tmB, ab, W, D, V, 1, pl->d.ldw, pl->d.ldw * V, 64, BK);
      ok = ok && encode_rows(&o.tmOut, GE_F32, part, pl->Dp, T, pl->slices, pl->Dp, pl->Dp * T, 32, 128);
      o.b_row0 = static_cast<int32_t>(v0);
      o.kb_split = pl->kb_split;
      o.splits = static_cast<int32_t>(ceil_div(ceil_div(n, BK), pl->kb_split));
      o.accumulate = v0 > 0;
      if (!ok) return GE_ERR_CUDA;
      go(launch_product(pl, pl->part, o, o.splits, s));
    }
  }
  if (dH) {
    SpreadParams dp{part, static_cast<uint16_t *>(dH), place, sc, pl->d.lddh, pl->Dp, static_cast<int32_t>(T),
                    static_cast<int32_t>(D), pl->slices, ab == GE_BF16};
    go(launch(reinterpret_cast<const void *>(xent_spread_kernel),
              static_cast<int>(std::min<int64_t>(ceil_div(T * ceil_div(D, 8), 256), spread_grid)), 256, 0, 1, &dp, s));
  }
  return ok ? GE_OK : GE_ERR_CUDA;
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
      desc->max_ctas < 0 || desc->reserved != 0 || desc->buffer_bytes < 0 || !std::isfinite(desc->logit_scale) ||
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
