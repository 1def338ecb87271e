// norm.cu -- the norms before and after a block, fused with its gate and
// residual scale, and their gradients (gemm_epi_norm_*).
//
//   y = x + alpha * gate * (N_post(b) * w_post),   h = N_pre(y) * w_pre
//
// A row is held whole by the threads that own it (8 consecutive columns per
// thread and chunk), so every tensor crosses the memory interface once: the
// forward pass reads x and b and writes y and h, the backward pass reads dy,
// dh, y and b and writes dx and db.  Statistics need no saved tensors: the
// rows they belong to are in registers anyway, so the backward pass computes
// them again.  Both passes are bound by memory: 4 and 6 elements per column
// of a row against a few fp32 operations each.
//
// Gradients, with u = N_pre(y), r_y its inverse divisor, n = N_post(b):
//   du = dh w_pre;   dN_pre = r_y (du - u mean(du u) [- mean(du) if centred])
//   t  = dy + dN_pre (the whole gradient of y) = dx
//   dn = alpha gate w_post t;  db = r_b (dn - n mean(dn n) [- mean(dn)])
//   dw_pre = sum dh u;  q_g = sum over group g's rows of t n;
//   dgate_g = alpha w_post q_g;  dw_post = alpha sum_g gate_g q_g
// so one sum over rows (q) serves both gate and w_post.  A unit of rows (one
// CTA, or a part of one when rows are narrow) sums its rows in registers and
// writes one partial row per sum; a second kernel adds the partials in a
// fixed order.  Units never straddle two gate groups unless they hold whole
// groups, in which case each group's dgate is finished by its unit.
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

using namespace ge;

namespace {

constexpr int kChunk = 8;        // columns a thread holds per chunk
constexpr int kMaxThreads = 1024;

struct NormParams {
  const void *x, *b, *gate, *w_post, *w_pre;
  void *y, *h;
  // gradients
  const void *dy, *dh, *yin;
  void *dx, *db, *dgate;
  float *part_pre, *part_post;  // [units][D]
  int64_t ldx, ldb, ldy, ldh;
  int64_t rows_per_gate;
  int32_t T, D, wt;
  int32_t pre, post;
  float eps_pre, eps_post, alpha, inv_d;
  int32_t row_threads;   // threads that share a row: a multiple of 32
  int32_t w_vec;         // rows of gate and the vectors are whole 16-byte units
  // units of the gradient pass
  int32_t units, rows_per_unit, units_per_group;  // units_per_group 0: a unit holds whole groups
};

template <int DT> struct Elem;
template <> struct Elem<GE_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <> struct Elem<GE_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<GE_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};

// 8 columns from `col` of a row of D; columns past the end read as 0.  kVec:
// the row starts on a 16-byte boundary (col is a multiple of 8).
template <int DT, bool kVec>
__device__ __forceinline__ void load8(const void *base, int64_t off, int col, int D, float (&v)[kChunk]) {
  using E = Elem<DT>;
  using T = typename E::T;
  const T *p = static_cast<const T *>(base) + off + col;
  if (kVec && col + kChunk <= D) {
    constexpr int kWords = kChunk * sizeof(T) / 16;
    union { uint4 w[kWords]; T e[kChunk]; } u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) u.w[i] = reinterpret_cast<const uint4 *>(p)[i];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = E::get(u.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = col + i < D ? E::get(p[i]) : 0.f;
  }
}

template <int DT, bool kVec>
__device__ __forceinline__ void store8(void *base, int64_t off, int col, int D, const float (&v)[kChunk]) {
  using E = Elem<DT>;
  using T = typename E::T;
  T *p = static_cast<T *>(base) + off + col;
  if (kVec && col + kChunk <= D) {
    constexpr int kWords = kChunk * sizeof(T) / 16;
    union { uint4 w[kWords]; T e[kChunk]; } u;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) u.e[i] = E::put(v[i]);
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = u.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (col + i < D) p[i] = E::put(v[i]);
  }
}

// weights and gates: their type is a uniform branch, not another kernel
__device__ __forceinline__ void loadw8(int wt, int vec, const void *base, int64_t off, int col, int D,
                                       float (&v)[kChunk]) {
  if (vec) {
    if (wt == GE_BF16) load8<GE_BF16, true>(base, off, col, D, v);
    else if (wt == GE_F16) load8<GE_F16, true>(base, off, col, D, v);
    else load8<GE_F32, true>(base, off, col, D, v);
  } else {
    if (wt == GE_BF16) load8<GE_BF16, false>(base, off, col, D, v);
    else if (wt == GE_F16) load8<GE_F16, false>(base, off, col, D, v);
    else load8<GE_F32, false>(base, off, col, D, v);
  }
}

__device__ __forceinline__ float getw(int wt, const void *base, int64_t i) {
  if (wt == GE_BF16) return Elem<GE_BF16>::get(static_cast<const __nv_bfloat16 *>(base)[i]);
  if (wt == GE_F16) return Elem<GE_F16>::get(static_cast<const __half *>(base)[i]);
  return static_cast<const float *>(base)[i];
}

__device__ __forceinline__ void putw(int wt, void *base, int64_t i, float v) {
  if (wt == GE_BF16) static_cast<__nv_bfloat16 *>(base)[i] = Elem<GE_BF16>::put(v);
  else if (wt == GE_F16) static_cast<__half *>(base)[i] = Elem<GE_F16>::put(v);
  else static_cast<float *>(base)[i] = v;
}

// Sums over the threads of a row.  One row per warp needs no shared memory;
// otherwise each warp leaves its sums in one of two buffers in turn (a buffer is
// written again only after the barrier of the next sum, which every reader
// of it has passed).
struct RowSum {
  float *buf;           // [2][warps of the CTA][4]
  int warps, warp0;     // warps of this row, the first of them
  int warp, lane, turn;
  template <int K>
  __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
    if (warps == 1) return;
    float *b = buf + turn * (kMaxThreads / 32) * 4;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) b[warp * 4 + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = warp0; w < warp0 + warps; ++w)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += b[w * 4 + k];
  }
};

// v[k][i] -= mean, with columns past the end kept at 0
template <int NV>
__device__ __forceinline__ void centre(float (&v)[NV][kChunk], float mean, int D, int t, int step) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int col = (t + k * step) * kChunk;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[k][i] = col + i < D ? v[k][i] - mean : 0.f;
  }
}

template <int NV>
__device__ __forceinline__ float sum_of(const float (&v)[NV][kChunk]) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) s += v[k][i];
  return s;
}

template <int NV>
__device__ __forceinline__ float dot_of(const float (&a)[NV][kChunk], const float (&b)[NV][kChunk]) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) s += a[k][i] * b[k][i];
  return s;
}

template <int NV>
__device__ __forceinline__ void scale(float (&v)[NV][kChunk], float f) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[k][i] *= f;
}

// v becomes N(v); returns the inverse divisor
template <int NV>
__device__ __forceinline__ float normalise(float (&v)[NV][kChunk], int kind, float eps, float inv_d, int D,
                                           int t, int step, RowSum &row_sum) {
  if (kind == GE_NORM_LAYER) {
    float m[1] = {sum_of(v)};
    row_sum(m);
    centre(v, m[0] * inv_d, D, t, step);
  }
  float s[1] = {dot_of(v, v)};
  row_sum(s);
  const float r = 1.f / sqrtf(s[0] * inv_d + eps);
  scale(v, r);
  return r;
}

template <int DT, int NV, bool kVec>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float buf[2 * (kMaxThreads / 32) * 4];
  griddep_wait();
  griddep_launch_dependents();
  const int per = p.row_threads, rows = blockDim.x / per;
  const int mine = threadIdx.x / per, t = threadIdx.x - mine * per;
  RowSum row_sum{buf, per / 32, mine * (per / 32), static_cast<int>(threadIdx.x >> 5),
                 static_cast<int>(threadIdx.x & 31), 0};
  for (int64_t first = int64_t(blockIdx.x) * rows; first < p.T; first += int64_t(gridDim.x) * rows) {
    const int64_t row = first + mine;
    const bool on = row < p.T;
    float y[NV][kChunk];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * per) * kChunk;
      load8<DT, kVec>(p.x, row * p.ldx, on ? col : p.D, p.D, y[k]);
    }
    if (p.b) {
      float b[NV][kChunk];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (t + k * per) * kChunk;
        load8<DT, kVec>(p.b, row * p.ldb, on ? col : p.D, p.D, b[k]);
      }
      if (p.post != GE_NORM_NONE)
        normalise(b, p.post, p.eps_post, p.inv_d, p.D, t, per, row_sum);
      const int64_t g = p.gate && on ? row / p.rows_per_gate : 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = on ? (t + k * per) * kChunk : p.D;
        if (p.w_post) {
          float w[kChunk];
          loadw8(p.wt, p.w_vec, p.w_post, 0, col, p.D, w);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) b[k][i] *= w[i];
        }
        if (p.gate) {
          float w[kChunk];
          loadw8(p.wt, p.w_vec, p.gate, g * p.D, col, p.D, w);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) b[k][i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) y[k][i] += p.alpha * b[k][i];
      }
    }
    if (p.y && on)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store8<DT, kVec>(p.y, row * p.ldy, (t + k * per) * kChunk, p.D, y[k]);
    if (p.h) {
      normalise(y, p.pre, p.eps_pre, p.inv_d, p.D, t, per, row_sum);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = on ? (t + k * per) * kChunk : p.D;
        if (p.w_pre) {
          float w[kChunk];
          loadw8(p.wt, p.w_vec, p.w_pre, 0, col, p.D, w);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) y[k][i] *= w[i];
        }
        if (on) store8<DT, kVec>(p.h, row * p.ldh, col, p.D, y[k]);
      }
    }
  }
}

// The rows of unit u, and the gate group its first row is in.
__device__ __forceinline__ void unit_rows(const NormParams &p, int u, int64_t &begin, int64_t &end) {
  begin = end = p.T;
  if (u >= p.units) return;
  if (p.units_per_group) {
    const int64_t g = u / p.units_per_group, s = u - g * p.units_per_group;
    begin = g * p.rows_per_gate + s * p.rows_per_unit;
    end = min(min(begin + p.rows_per_unit, (g + 1) * p.rows_per_gate), int64_t(p.T));
    begin = min(begin, end);
  } else {
    begin = int64_t(u) * p.rows_per_unit;
    end = min(begin + p.rows_per_unit, int64_t(p.T));
  }
}

template <int DT, int NV, bool kVec>
__global__ void __launch_bounds__(kMaxThreads) norm_grad_kernel(const __grid_constant__ NormParams p) {
  __shared__ float buf[2 * (kMaxThreads / 32) * 4];
  griddep_wait();
  griddep_launch_dependents();
  const int per = p.row_threads, lanes = blockDim.x / per;
  const int mine = threadIdx.x / per, t = threadIdx.x - mine * per;
  RowSum row_sum{buf, per / 32, mine * (per / 32), static_cast<int>(threadIdx.x >> 5),
                 static_cast<int>(threadIdx.x & 31), 0};
  const int u = blockIdx.x * lanes + mine;
  int64_t begin, end;
  unit_rows(p, u, begin, end);
  float acc_pre[NV][kChunk], acc_post[NV][kChunk];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) acc_pre[k][i] = acc_post[k][i] = 0.f;
  float acc_gate[NV][kChunk];  // whole groups: the current group's q
  const bool whole = p.gate && p.units_per_group == 0;
  if (whole)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) acc_gate[k][i] = 0.f;

  for (int r = 0; r < p.rows_per_unit; ++r) {  // every thread: row sums hold barriers
    const int64_t row = begin + r;
    const bool on = row < end;
    float y[NV][kChunk], d[NV][kChunk];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = on ? (t + k * per) * kChunk : p.D;
      load8<DT, kVec>(p.yin, row * p.ldy, col, p.D, y[k]);
      load8<DT, kVec>(p.dh, row * p.ldh, col, p.D, d[k]);
    }
    const float ry = normalise(y, p.pre, p.eps_pre, p.inv_d, p.D, t, per, row_sum);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = on ? (t + k * per) * kChunk : p.D;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) acc_pre[k][i] += d[k][i] * y[k][i];
      if (p.w_pre) {
        float w[kChunk];
        loadw8(p.wt, p.w_vec, p.w_pre, 0, col, p.D, w);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) d[k][i] *= w[i];
      }
    }
    float s[2] = {dot_of(d, y), p.pre == GE_NORM_LAYER ? sum_of(d) : 0.f};
    row_sum(s);
    s[0] *= p.inv_d;
    s[1] *= p.inv_d;
    // d becomes the whole gradient of y
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = on ? (t + k * per) * kChunk : p.D;
      float g[kChunk];
      if (p.dy) load8<DT, kVec>(p.dy, row * p.ldy, col, p.D, g);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        d[k][i] = (col + i < p.D ? ry * (d[k][i] - s[1] - y[k][i] * s[0]) : 0.f) + (p.dy ? g[i] : 0.f);
    }
    if (p.b) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        load8<DT, kVec>(p.b, row * p.ldb, on ? (t + k * per) * kChunk : p.D, p.D, y[k]);
    }
    if (on)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store8<DT, kVec>(p.dx, row * p.ldx, (t + k * per) * kChunk, p.D, d[k]);
    if (!p.b) continue;
    float rb = 1.f;
    if (p.post != GE_NORM_NONE) rb = normalise(y, p.post, p.eps_post, p.inv_d, p.D, t, per, row_sum);
    const int64_t g = p.gate && on ? row / p.rows_per_gate : 0;
    const bool last = whole && on && (row + 1 == end || (row + 1) % p.rows_per_gate == 0);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = on ? (t + k * per) * kChunk : p.D;
      float gw[kChunk];
      if (p.gate) loadw8(p.wt, p.w_vec, p.gate, g * p.D, col, p.D, gw);
      float pw[kChunk];
      if (p.w_post) loadw8(p.wt, p.w_vec, p.w_post, 0, col, p.D, pw);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const float q = d[k][i] * y[k][i];
        if (whole) acc_gate[k][i] += q;
        else acc_post[k][i] += q;
        d[k][i] *= p.alpha;
        if (p.gate) d[k][i] *= gw[i];
        if (p.w_post) d[k][i] *= pw[i];
      }
      if (last) {
        // the group's last row: its gate's gradient is complete
        float o[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          acc_post[k][i] += gw[i] * acc_gate[k][i];
          o[i] = p.alpha * acc_gate[k][i] * (p.w_post ? pw[i] : 1.f);
          acc_gate[k][i] = 0.f;
        }
        if (p.dgate)
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (col + i < p.D) putw(p.wt, p.dgate, g * p.D + col + i, o[i]);
      }
    }
    if (p.post != GE_NORM_NONE) {
      float s2[2] = {dot_of(d, y), p.post == GE_NORM_LAYER ? sum_of(d) : 0.f};
      row_sum(s2);
      s2[0] *= p.inv_d;
      s2[1] *= p.inv_d;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) d[k][i] = rb * (d[k][i] - s2[1] - y[k][i] * s2[0]);
    }
    if (p.db && on)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store8<DT, kVec>(p.db, row * p.ldb, (t + k * per) * kChunk, p.D, d[k]);
  }
  if (u < p.units) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * per) * kChunk;
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col + i < p.D) {
          p.part_pre[int64_t(u) * p.D + col + i] = acc_pre[k][i];
          if (p.part_post) p.part_post[int64_t(u) * p.D + col + i] = acc_post[k][i];
        }
    }
  }
}

// Adds the units' partial rows.  grid.y 0: dw_pre and dw_post; grid.y 1 + g: the
// gate of group g (units that hold part of one group).  Each of the 32 threads
// of a column adds every 32nd unit, then the 32 sums are added in order.
struct SumParams {
  const float *part_pre, *part_post;
  const void *gate, *w_post;
  void *dgate, *dw_post, *dw_pre;
  float alpha;
  int32_t D, wt, units, units_per_group;
};

constexpr int kSumCols = 32, kSumLanes = 32;

__global__ void __launch_bounds__(kSumCols *kSumLanes) norm_sum_kernel(const __grid_constant__ SumParams p) {
  __shared__ float part[2][kSumLanes][kSumCols + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int col = blockIdx.x * kSumCols + threadIdx.x, lane = threadIdx.y;
  const bool on = col < p.D;
  float a = 0.f, b = 0.f;
  if (blockIdx.y == 0) {
    for (int u = lane; on && u < p.units; u += kSumLanes) {
      const int64_t at = int64_t(u) * p.D + col;
      if (p.dw_pre) a += p.part_pre[at];
      if (p.dw_post) {
        const float q = p.part_post[at];
        // units of whole groups have their gates in the sum already
        b += p.gate && p.units_per_group ? q * getw(p.wt, p.gate, int64_t(u / p.units_per_group) * p.D + col) : q;
      }
    }
  } else {
    const int g = blockIdx.y - 1;
    for (int s = lane; on && s < p.units_per_group; s += kSumLanes) {
      const int u = g * p.units_per_group + s;
      a += p.part_post[int64_t(u) * p.D + col];
    }
  }
  part[0][lane][threadIdx.x] = a;
  part[1][lane][threadIdx.x] = b;
  __syncthreads();
  if (lane || !on) return;
  a = b = 0.f;
  for (int l = 0; l < kSumLanes; ++l) {
    a += part[0][l][threadIdx.x];
    b += part[1][l][threadIdx.x];
  }
  if (blockIdx.y == 0) {
    if (p.dw_pre) putw(p.wt, p.dw_pre, col, a);
    if (p.dw_post) putw(p.wt, p.dw_post, col, p.alpha * b);
  } else {
    const float w = p.w_post ? getw(p.wt, p.w_post, col) : 1.f;
    putw(p.wt, p.dgate, int64_t(blockIdx.y - 1) * p.D + col, p.alpha * w * a);
  }
}

template <int NV, bool kVec>
const void *pick_type(int dt, bool grad) {
  if (grad)
    return dt == GE_F16    ? reinterpret_cast<const void *>(norm_grad_kernel<GE_F16, NV, kVec>)
           : dt == GE_BF16 ? reinterpret_cast<const void *>(norm_grad_kernel<GE_BF16, NV, kVec>)
                           : reinterpret_cast<const void *>(norm_grad_kernel<GE_F32, NV, kVec>);
  return dt == GE_F16    ? reinterpret_cast<const void *>(norm_kernel<GE_F16, NV, kVec>)
         : dt == GE_BF16 ? reinterpret_cast<const void *>(norm_kernel<GE_BF16, NV, kVec>)
                         : reinterpret_cast<const void *>(norm_kernel<GE_F32, NV, kVec>);
}

const void *pick_kernel(int dt, int nv, bool vec, bool grad) {
  if (nv == 1) return vec ? pick_type<1, true>(dt, grad) : pick_type<1, false>(dt, grad);
  if (nv == 2) return vec ? pick_type<2, true>(dt, grad) : pick_type<2, false>(dt, grad);
  return vec ? pick_type<4, true>(dt, grad) : pick_type<4, false>(dt, grad);
}

bool valid_type(int t) { return t == GE_F16 || t == GE_BF16 || t == GE_F32; }
int64_t size_of(int t) { return t == GE_F32 ? 4 : 2; }

// How a row is shared out: chunks of 8 columns per thread and threads per row.
struct RowShape {
  const void *fn = nullptr;
  int nv = 1, row_threads = 32, threads = 32, grid = 1;
};

cudaError_t launch(const void *fn, dim3 grid, dim3 block, void *params, cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void *args[] = {params};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

struct gemm_epi_norm_plan {
  int64_t T = 0, D = 0;
  ge_norm_desc d{};
  int sms = 0;
  bool vec = false;
  RowShape fwd, bwd;
  NormParams p{};
};

namespace {

bool shape_of(const gemm_epi_norm_plan *pl, bool grad, RowShape *out) {
  const int chunks = static_cast<int>(ceil_div(pl->D, kChunk));
  RowShape r;
  // one chunk per thread while a row fits 512 threads, then more
  r.nv = chunks <= 512 ? 1 : (chunks <= 2048 ? 2 : 4);
  r.row_threads = static_cast<int>(round_up(ceil_div(chunks, r.nv), 32));
  const int rows = std::max(1, 256 / r.row_threads);
  r.threads = r.row_threads * rows;
  r.fn = pick_kernel(pl->d.x, r.nv, pl->vec, grad);
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, r.fn, r.threads, 0) != cudaSuccess || per_sm < 1) {
    cudaGetLastError();
    return false;
  }
  r.grid = static_cast<int>(std::min<int64_t>(ceil_div(pl->T, rows), int64_t(pl->sms) * per_sm));
  *out = r;
  return true;
}

// Units of the gradient pass: as many as the GPU holds at once, rounded so that
// a unit stays inside a gate group or holds whole ones.
void share_rows(gemm_epi_norm_plan *pl) {
  NormParams &p = pl->p;
  const RowShape &r = pl->bwd;
  const int64_t lanes = r.threads / r.row_threads;
  int64_t want = ceil_div(pl->T, std::min<int64_t>(pl->T, int64_t(r.grid) * lanes));  // rows per unit
  const int64_t rpg = pl->d.rows_per_gate ? std::min<int64_t>(pl->d.rows_per_gate, pl->T) : pl->T;
  const int64_t groups = ceil_div(pl->T, rpg);
  if (rpg <= want && pl->d.rows_per_gate) {
    p.rows_per_unit = static_cast<int32_t>(want / rpg * rpg);
    p.units_per_group = 0;
    p.units = static_cast<int32_t>(ceil_div(pl->T, p.rows_per_unit));
  } else {
    p.units_per_group = static_cast<int32_t>(ceil_div(rpg, want));
    p.rows_per_unit = static_cast<int32_t>(ceil_div(rpg, p.units_per_group));
    p.units_per_group = static_cast<int32_t>(ceil_div(rpg, p.rows_per_unit));
    p.units = static_cast<int32_t>(groups * p.units_per_group);
  }
}

int check_ptr(const void *p) { return !p ? GE_ERR_MISSING_ARG : (is_aligned16(p) ? GE_OK : GE_ERR_MISALIGNED); }
int check_opt(const void *p) { return !p || is_aligned16(p) ? GE_OK : GE_ERR_MISALIGNED; }

// gate, w_post and w_pre as both passes take them
int check_block(const gemm_epi_norm_plan *pl, const void *b, const void *gate, const void *w_post,
                const void *w_pre) {
  for (const void *q : {b, gate, w_post, w_pre})
    if (check_opt(q) != GE_OK) return GE_ERR_MISALIGNED;
  if (!b) return gate || w_post ? GE_ERR_INVALID : GE_OK;
  if (pl->d.rows_per_gate && !gate) return GE_ERR_MISSING_ARG;
  if (!pl->d.rows_per_gate && gate) return GE_ERR_INVALID;
  if (pl->d.post == GE_NORM_NONE && w_post) return GE_ERR_INVALID;
  return GE_OK;
}

}  // namespace

extern "C" {

int gemm_epi_norm_plan_create(gemm_epi_norm_plan **plan, int64_t T, int64_t D, const ge_norm_desc *desc) {
  if (!plan) return GE_ERR_INVALID;
  *plan = nullptr;
  if (!desc) return GE_ERR_INVALID;
  if (!valid_type(desc->x) || !valid_type(desc->w)) return GE_ERR_UNSUPPORTED;
  if (desc->pre != GE_NORM_RMS && desc->pre != GE_NORM_LAYER) return GE_ERR_INVALID;
  if (desc->post < GE_NORM_NONE || desc->post > GE_NORM_LAYER) return GE_ERR_INVALID;
  if (!(desc->eps_pre >= 0.f) || !(desc->eps_post >= 0.f) || !std::isfinite(desc->eps_pre) ||
      !std::isfinite(desc->eps_post) || !std::isfinite(desc->alpha) || desc->reserved != 0 ||
      desc->rows_per_gate < 0)
    return GE_ERR_INVALID;
  if (T <= 0 || D <= 0 || D > GE_NORM_MAX_D || T > (int64_t(1) << 31) - 1) return GE_ERR_SHAPE;
  ge_norm_desc d = *desc;
  for (int64_t *ld : {&d.ldx, &d.ldb, &d.ldy, &d.ldh}) {
    if (*ld == 0) *ld = D;
    if (*ld < D || *ld > (int64_t(1) << 31) - 1) return GE_ERR_SHAPE;
  }
  gemm_epi_norm_plan *pl = new (std::nothrow) gemm_epi_norm_plan();
  if (!pl) return GE_ERR_INVALID;
  pl->T = T;
  pl->D = D;
  pl->d = d;
  const int64_t es = size_of(d.x);
  pl->vec = true;
  for (int64_t ld : {d.ldx, d.ldb, d.ldy, d.ldh}) pl->vec = pl->vec && (ld * es) % 16 == 0;
  int dev = 0, smem = 0;
  int st = current_device(&dev, &pl->sms, &smem);
  if (st == GE_OK && (!shape_of(pl, false, &pl->fwd) || !shape_of(pl, true, &pl->bwd))) st = GE_ERR_CUDA;
  if (st != GE_OK) {
    delete pl;
    return st;
  }
  NormParams &p = pl->p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  p.ldx = d.ldx;
  p.ldb = d.ldb;
  p.ldy = d.ldy;
  p.ldh = d.ldh;
  // without a gate, one group of all rows
  p.rows_per_gate = d.rows_per_gate ? std::min<int64_t>(d.rows_per_gate, T) : T;
  p.T = static_cast<int32_t>(T);
  p.D = static_cast<int32_t>(D);
  p.wt = d.w;
  p.pre = d.pre;
  p.post = d.post;
  p.eps_pre = d.eps_pre;
  p.eps_post = d.eps_post;
  p.alpha = d.alpha;
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(D));
  p.w_vec = (D * size_of(d.w)) % 16 == 0;
  share_rows(pl);
  *plan = pl;
  return GE_OK;
}

void gemm_epi_norm_plan_destroy(gemm_epi_norm_plan *plan) { delete plan; }

size_t gemm_epi_norm_workspace_bytes(const gemm_epi_norm_plan *pl) {
  if (!pl) return 0;
  return 2u * sizeof(float) * static_cast<size_t>(pl->p.units) * static_cast<size_t>(pl->D);
}

int gemm_epi_norm_run(gemm_epi_norm_plan *pl, const void *x, const void *b, const void *gate,
                      const void *w_post, const void *w_pre, void *y, void *h, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  int st = check_ptr(x);
  if (st == GE_OK) st = check_block(pl, b, gate, w_post, w_pre);
  if (st != GE_OK) return st;
  if (!y && !h) return GE_ERR_MISSING_ARG;
  if (check_opt(y) != GE_OK || check_opt(h) != GE_OK) return GE_ERR_MISALIGNED;
  const ge_norm_desc &d = pl->d;
  // in place: a row is read before it is written only where the rows coincide
  if (y && y == h) return GE_ERR_INVALID;
  if ((y == x && d.ldy != d.ldx) || (b && y == b && d.ldy != d.ldb) || (h == x && d.ldh != d.ldx) ||
      (b && h == b && d.ldh != d.ldb))
    return GE_ERR_INVALID;
  NormParams p = pl->p;
  p.x = x;
  p.b = b;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.y = y;
  p.h = h;
  p.row_threads = pl->fwd.row_threads;
  const cudaError_t e = launch(pl->fwd.fn, dim3(pl->fwd.grid), dim3(pl->fwd.threads), &p,
                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GE_OK : GE_ERR_CUDA;
}

int gemm_epi_norm_grad(gemm_epi_norm_plan *pl, const void *dy, const void *dh, const void *y,
                       const void *b, const void *gate, const void *w_post, const void *w_pre,
                       void *dx, void *db, void *dgate, void *dw_post, void *dw_pre,
                       void *workspace, size_t workspace_bytes, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  for (const void *q : {dh, y, static_cast<const void *>(dx)}) {
    const int st = check_ptr(q);
    if (st != GE_OK) return st;
  }
  int st = check_block(pl, b, gate, w_post, w_pre);
  if (st != GE_OK) return st;
  for (const void *q : {dy, static_cast<const void *>(db), static_cast<const void *>(dgate),
                        static_cast<const void *>(dw_post), static_cast<const void *>(dw_pre)})
    if (check_opt(q) != GE_OK) return GE_ERR_MISALIGNED;
  // a gradient of something that takes no part
  if ((!b && (db || dgate || dw_post)) || (!gate && dgate) || (!w_post && dw_post) || (!w_pre && dw_pre))
    return GE_ERR_INVALID;
  const ge_norm_desc &d = pl->d;
  if (dx == db || (dx == dy && d.ldx != d.ldy) || (dx == dh && d.ldx != d.ldh) ||
      (db && db == dh && d.ldb != d.ldh))
    return GE_ERR_INVALID;
  if (!workspace || !is_aligned16(workspace) || workspace_bytes < gemm_epi_norm_workspace_bytes(pl))
    return GE_ERR_WORKSPACE;
  NormParams p = pl->p;
  p.dy = dy;
  p.dh = dh;
  p.yin = y;
  p.b = b;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.dx = dx;
  p.db = db;
  p.dgate = dgate;
  p.row_threads = pl->bwd.row_threads;
  p.part_pre = static_cast<float *>(workspace);
  p.part_post = b ? p.part_pre + static_cast<size_t>(p.units) * static_cast<size_t>(pl->D) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int lanes = pl->bwd.threads / pl->bwd.row_threads;
  const int grid = static_cast<int>(ceil_div(p.units, lanes));
  if (launch(pl->bwd.fn, dim3(grid), dim3(pl->bwd.threads), &p, s) != cudaSuccess) return GE_ERR_CUDA;
  const bool gates = dgate && p.units_per_group;
  if (!dw_pre && !dw_post && !gates) return GE_OK;
  SumParams q;
  std::memset(static_cast<void *>(&q), 0, sizeof(q));
  q.part_pre = p.part_pre;
  q.part_post = p.part_post;
  q.gate = gate;
  q.w_post = w_post;
  q.dgate = dgate;
  q.dw_post = dw_post;
  q.dw_pre = dw_pre;
  q.alpha = p.alpha;
  q.D = p.D;
  q.wt = p.wt;
  q.units = p.units;
  q.units_per_group = p.units_per_group;
  const int groups = gates ? p.units / p.units_per_group : 0;
  const cudaError_t e = launch(reinterpret_cast<const void *>(norm_sum_kernel),
                               dim3(static_cast<unsigned>(ceil_div(p.D, kSumCols)), static_cast<unsigned>(1 + groups)),
                               dim3(kSumCols, kSumLanes), &q, s);
  return e == cudaSuccess ? GE_OK : GE_ERR_CUDA;
}

}  // extern "C"
