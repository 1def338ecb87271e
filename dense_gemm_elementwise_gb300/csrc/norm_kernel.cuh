// norm_kernel.cuh -- the norms before and after a block, fused with its gate and
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
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_epi.h"
#include "norm.h"
#include "ptx.cuh"

namespace ge {


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

// Which columns a thread holds.  Rows of whole 16-byte units: 8 in a run, moved
// 16 bytes at a time.  Other rows: every row_threads-th column, so that the
// threads of a warp read neighbouring elements (8 in a run would have each
// load touch four times the cache lines; 3001 x 1111 fp16 took 20.7 us so).
template <bool kVec>
struct Columns {
  int t, per;
  __device__ __forceinline__ int operator()(int k, int i) const {
    return kVec ? (t + k * per) * kChunk + i : (k * kChunk + i) * per + t;
  }
};

template <int DT, int NV, bool kVec>
__device__ __forceinline__ void load_row(const void *base, int64_t off, const Columns<kVec> &col, int D, bool on,
                                         float (&v)[NV][kChunk]) {
  using E = Elem<DT>;
  const typename E::T *p = static_cast<const typename E::T *>(base) + off;
  if (!on) D = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[k][i] = col(k, i) < D ? E::get(p[col(k, i)]) : 0.f;
}

template <int DT, int NV, bool kVec>
__device__ __forceinline__ void store_row(void *base, int64_t off, const Columns<kVec> &col, int D,
                                          const float (&v)[NV][kChunk]) {
  using E = Elem<DT>;
  using T = typename E::T;
  T *p = static_cast<T *>(base) + off;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (kVec && col(k, 0) + kChunk <= D) {
      constexpr int kWords = kChunk * sizeof(T) / 16;
      union { uint4 w[kWords]; T e[kChunk]; } u;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) u.e[i] = E::put(v[k][i]);
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4 *>(p + col(k, 0))[i] = u.w[i];
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col(k, i) < D) p[col(k, i)] = E::put(v[k][i]);
    }
  }
}

// weights and gates: their type is a uniform branch, not another kernel
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

// w[k][i] = base[off + column], 1 where base is NULL, 0 past the end
template <int NV, bool kVec>
__device__ __forceinline__ void load_w(const NormParams &p, const void *base, int64_t off, const Columns<kVec> &col,
                                       float (&w)[NV][kChunk]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (kVec && base && p.w_vec && col(k, 0) < p.D) {
      if (p.wt == GE_F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off + col(k, 0));
        const float4 a = q[0], b = col(k, 4) < p.D ? q[1] : make_float4(0.f, 0.f, 0.f, 0.f);
        w[k][0] = a.x, w[k][1] = a.y, w[k][2] = a.z, w[k][3] = a.w;
        w[k][4] = b.x, w[k][5] = b.y, w[k][6] = b.z, w[k][7] = b.w;
      } else {
        union { uint4 v; __half h[8]; __nv_bfloat16 b[8]; } u;
        u.v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off + col(k, 0));
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          w[k][i] = p.wt == GE_F16 ? __half2float(u.h[i]) : __bfloat162float(u.b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        w[k][i] = col(k, i) < p.D ? (base ? getw(p.wt, base, off + col(k, i)) : 1.f) : 0.f;
    }
  }
}

// Shared memory of a thread's own: `threads` 16-byte words side by side, so
// that a warp's accesses are free of conflicts, and no barrier: nobody else
// reads them.
struct Own {
  uint4 *base;   // this thread's first word
  int threads;
  template <int NV>
  __device__ __forceinline__ void put(const float (&w)[NV][kChunk]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<float4 *>(base)[(2 * k + j) * threads] =
            make_float4(w[k][4 * j], w[k][4 * j + 1], w[k][4 * j + 2], w[k][4 * j + 3]);
  }
  // the same factors, multiplied into v
  template <int NV>
  __device__ __forceinline__ void times(float (&v)[NV][kChunk]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 f = reinterpret_cast<const float4 *>(base)[(2 * k + j) * threads];
        v[k][4 * j] *= f.x, v[k][4 * j + 1] *= f.y, v[k][4 * j + 2] *= f.z, v[k][4 * j + 3] *= f.w;
      }
  }
};

// A ring of rows on their way from memory (cp.async into the thread's own
// words): `ahead` rows of NA tensors each.  Rows that are not whole 16-byte
// units are read when they are wanted.
template <int DT, int NV, bool kVec, int NA>
struct Ring {
  static constexpr int kWords = kChunk * sizeof(typename Elem<DT>::T) / 16;  // of one tensor's chunk
  static constexpr int kRow = NA * NV * kWords;  // 16-byte words of a thread per row
  uint4 *base;
  int threads, ahead, D;
  Columns<kVec> col;

  __device__ __forceinline__ void issue(int slot, int a, const void *src, int64_t off, bool on) const {
    if constexpr (kVec) {
      using T = typename Elem<DT>::T;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          constexpr int kPer = 16 / sizeof(T);
          const int c = col(k, 0) + j * kPer;
          const int left = on && src ? min(max(D - c, 0), kPer) * static_cast<int>(sizeof(T)) : 0;
          const T *p = left ? static_cast<const T *>(src) + off + c : static_cast<const T *>(src);
          const uint32_t dst = smem_u32(base + (slot * kRow + (a * NV + k) * kWords + j) * threads);
          if (left > 0)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(left) : "memory");
          else
            *reinterpret_cast<uint4 *>(base + (slot * kRow + (a * NV + k) * kWords + j) * threads) =
                make_uint4(0u, 0u, 0u, 0u);
        }
    }
  }
  __device__ __forceinline__ void commit() const {
    if constexpr (kVec) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the oldest row of the ring has landed
  __device__ __forceinline__ void wait() const {
    if constexpr (kVec) {
      if (ahead == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (ahead == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  }
  __device__ __forceinline__ void get(int slot, int a, const void *src, int64_t off, bool on,
                                      float (&v)[NV][kChunk]) const {
    if constexpr (kVec) {
      using T = typename Elem<DT>::T;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        union { uint4 w[kWords]; T e[kChunk]; } u;
#pragma unroll
        for (int j = 0; j < kWords; ++j) u.w[j] = base[(slot * kRow + (a * NV + k) * kWords + j) * threads];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[k][i] = Elem<DT>::get(u.e[i]);
      }
    } else {
      load_row<DT, NV, kVec>(src, off, col, D, on && src, v);
    }
  }
};

// Sums over the threads of a row.  A row of at most a warp needs no shared
// memory; otherwise each warp leaves its sums in one of two buffers in turn (a
// buffer is written again only after the barrier of the next sum, which every
// reader of it has passed).  The barrier is the row's own.
struct RowSum {
  float4 *buf;          // this row's [2][warps]
  int per, warps, warp, lane, id, turn;
  template <int K>
  __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      if (s < per)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
    if (warps <= 1) return;
    float4 *b = buf + turn * warps;
    turn ^= 1;
    if (lane == 0) b[warp] = make_float4(v[0], K > 1 ? v[K > 1 ? 1 : 0] : 0.f, 0.f, 0.f);
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(per) : "memory");
    // 32 lanes add up to 32 warps' sums
    float4 f = lane < warps ? b[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      f.x += __shfl_xor_sync(0xffffffffu, f.x, s);
      if (K > 1) f.y += __shfl_xor_sync(0xffffffffu, f.y, s);
    }
    v[0] = f.x;
    if (K > 1) v[K > 1 ? 1 : 0] = f.y;
  }
};

// v -= mean, with columns past the end kept at 0
template <int NV, bool kVec>
__device__ __forceinline__ void centre(float (&v)[NV][kChunk], float mean, int D, const Columns<kVec> &col) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[k][i] = col(k, i) < D ? v[k][i] - mean : 0.f;
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

// v becomes N(v); returns the inverse divisor
template <int NV, bool kVec>
__device__ __forceinline__ float normalise(float (&v)[NV][kChunk], int kind, float eps, float inv_d, int D,
                                           const Columns<kVec> &col, RowSum &row_sum) {
  if (kind == GE_NORM_LAYER) {
    float m[1] = {sum_of(v)};
    row_sum(m);
    centre(v, m[0] * inv_d, D, col);
  }
  float s[1] = {dot_of(v, v)};
  row_sum(s);
  const float r = 1.f / sqrtf(s[0] * inv_d + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[k][i] *= r;
  return r;
}

// A CTA's share of its shared memory: the rows' sums, then (keep_w) the
// factors w_pre and alpha gate w_post of each thread's columns, then the ring.
template <bool kVec>
struct Place {
  int per, mine, t;
  __device__ __forceinline__ Place(int row_threads)
      : per(row_threads), mine(threadIdx.x / row_threads), t(threadIdx.x - mine * row_threads) {}
  __device__ __forceinline__ Columns<kVec> columns() const { return Columns<kVec>{t, per}; }
  __device__ __forceinline__ RowSum row_sum(uint8_t *smem) const {
    const int warps = per / 32;
    return RowSum{reinterpret_cast<float4 *>(smem) + 2 * mine * warps, per, warps, t >> 5,
                  static_cast<int>(threadIdx.x & 31), 1 + mine, 0};
  }
};

// v *= alpha gate w_post for the rows of gate group g (kept: `at` is the group the kept factors are for)
template <int NV, bool kVec>
__device__ __forceinline__ void times_post(const NormParams &p, const Columns<kVec> &col, const Own &own, int64_t g,
                                           int64_t &at, float (&v)[NV][kChunk]) {
  if (p.keep_w && at == g) {
    own.times(v);
    return;
  }
  float f[NV][kChunk], w[NV][kChunk];
  load_w<NV, kVec>(p, p.gate, p.gate ? g * p.D : 0, col, f);
  load_w<NV, kVec>(p, p.w_post, 0, col, w);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      f[k][i] *= p.alpha * w[k][i];
      v[k][i] *= f[k][i];
    }
  if (p.keep_w) own.put(f);
  at = g;
}

template <int NV, bool kVec>
__device__ __forceinline__ void times_pre(const NormParams &p, const Columns<kVec> &col, const Own &own,
                                          float (&v)[NV][kChunk]) {
  if (!p.w_pre) return;
  if (p.keep_w) {
    own.times(v);
    return;
  }
  float w[NV][kChunk];
  load_w<NV, kVec>(p, p.w_pre, 0, col, w);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[k][i] *= w[k][i];
}

template <int DT, int NV, bool kVec>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Place<kVec> pl(p.row_threads);
  const int rows = blockDim.x / pl.per;
  const Columns<kVec> col = pl.columns();
  RowSum row_sum = pl.row_sum(smem);
  uint4 *words = reinterpret_cast<uint4 *>(smem + kSumBytes) + threadIdx.x;
  const int n = blockDim.x;
  const Own own_pre{words, n}, own_post{words + 2 * NV * n, n};
  const Ring<DT, NV, kVec, 2> ring{words + (p.keep_w ? 4 * NV * n : 0), n, p.ahead, p.D, col};
  const int64_t step = int64_t(gridDim.x) * rows;
  int64_t row = int64_t(blockIdx.x) * rows + pl.mine;
  griddep_wait();
  griddep_launch_dependents();
  for (int s = 0; s < p.ahead - 1; ++s) {
    const int64_t r = row + s * step;
    ring.issue(s, 0, p.x, r * p.ldx, r < p.T);
    ring.issue(s, 1, p.b, r * p.ldb, r < p.T);
    ring.commit();
  }
  if (p.keep_w && p.w_pre) {
    float w[NV][kChunk];
    load_w<NV, kVec>(p, p.w_pre, 0, col, w);
    own_pre.put(w);
  }
  int64_t at = -1;
  int slot = 0, next = p.ahead - 1;
  // rows of a CTA that share warps stay together: they leave the loop at once
  for (int64_t first = int64_t(blockIdx.x) * rows; first < p.T; first += step, row += step) {
    const bool on = row < p.T;
    {
      const int64_t r = row + (p.ahead - 1) * step;
      ring.issue(next, 0, p.x, r * p.ldx, r < p.T);
      ring.issue(next, 1, p.b, r * p.ldb, r < p.T);
      ring.commit();
      if (++next == p.ahead) next = 0;
    }
    ring.wait();
    float y[NV][kChunk];
    if (p.b) {
      float b[NV][kChunk];
      ring.get(slot, 1, p.b, row * p.ldb, on, b);
      if (p.post != GE_NORM_NONE) normalise(b, p.post, p.eps_post, p.inv_d, p.D, col, row_sum);
      times_post<NV, kVec>(p, col, own_post, p.gate && on ? row / p.rows_per_gate : 0, at, b);
      ring.get(slot, 0, p.x, row * p.ldx, on, y);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) y[k][i] += b[k][i];
    } else {
      ring.get(slot, 0, p.x, row * p.ldx, on, y);
    }
    if (++slot == p.ahead) slot = 0;
    if (p.y && on) store_row<DT, NV, kVec>(p.y, row * p.ldy, col, p.D, y);
    if (p.h) {
      normalise(y, p.pre, p.eps_pre, p.inv_d, p.D, col, row_sum);
      times_pre<NV, kVec>(p, col, own_pre, y);
      if (on) store_row<DT, NV, kVec>(p.h, row * p.ldh, col, p.D, y);
    }
  }
}

// The rows of unit u.
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

// kWhole: a unit holds whole gate groups
template <int DT, int NV, bool kVec, bool kWhole>
__global__ void __launch_bounds__(kMaxThreads) norm_grad_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Place<kVec> pl(p.row_threads);
  const Columns<kVec> col = pl.columns();
  RowSum row_sum = pl.row_sum(smem);
  uint4 *words = reinterpret_cast<uint4 *>(smem + kSumBytes) + threadIdx.x;
  const int n = blockDim.x;
  const Own own_pre{words, n}, own_post{words + 2 * NV * n, n};
  const Ring<DT, NV, kVec, 4> ring{words + (p.keep_w ? 4 * NV * n : 0), n, p.ahead, p.D, col};
  const int u = blockIdx.x * (n / pl.per) + pl.mine;
  int64_t row, end;
  unit_rows(p, u, row, end);
  griddep_wait();
  griddep_launch_dependents();
  auto fetch = [&](int slot, int64_t r) {
    ring.issue(slot, 0, p.yin, r * p.ldy, r < end);
    ring.issue(slot, 1, p.dh, r * p.ldh, r < end);
    ring.issue(slot, 2, p.dy, r * p.ldy, r < end);
    ring.issue(slot, 3, p.b, r * p.ldb, r < end);
    ring.commit();
  };
  for (int s = 0; s < p.ahead - 1; ++s) fetch(s, row + s);
  if (p.keep_w && p.w_pre) {
    float w[NV][kChunk];
    load_w<NV, kVec>(p, p.w_pre, 0, col, w);
    own_pre.put(w);
  }
  float acc_pre[NV][kChunk], acc_post[NV][kChunk];
  float acc_gate[kWhole ? NV : 1][kChunk];  // whole groups: the current group's q
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      acc_pre[k][i] = acc_post[k][i] = 0.f;
      if (kWhole) acc_gate[k][i] = 0.f;
    }
  int64_t at = -1;
  int slot = 0, next = p.ahead - 1;
  for (int r = 0; r < p.rows_per_unit; ++r, ++row) {  // every thread: row sums hold barriers
    const bool on = row < end;
    fetch(next, row + p.ahead - 1);
    if (++next == p.ahead) next = 0;
    ring.wait();
    float y[NV][kChunk], d[NV][kChunk];
    ring.get(slot, 0, p.yin, row * p.ldy, on, y);
    ring.get(slot, 1, p.dh, row * p.ldh, on, d);
    const float ry = normalise(y, p.pre, p.eps_pre, p.inv_d, p.D, col, row_sum);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) acc_pre[k][i] += d[k][i] * y[k][i];
    times_pre<NV, kVec>(p, col, own_pre, d);
    float s[2] = {dot_of(d, y), p.pre == GE_NORM_LAYER ? sum_of(d) : 0.f};
    row_sum(s);
    s[0] *= p.inv_d;
    s[1] *= p.inv_d;
    // d becomes the whole gradient of y
    {
      float g[NV][kChunk];
      ring.get(slot, 2, p.dy, row * p.ldy, on && p.dy, g);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          d[k][i] = (col(k, i) < p.D ? ry * (d[k][i] - s[1] - y[k][i] * s[0]) : 0.f) + g[k][i];
    }
    if (p.b) ring.get(slot, 3, p.b, row * p.ldb, on, y);  // read before dx is written: it may be in b's place
    if (++slot == p.ahead) slot = 0;
    if (on) store_row<DT, NV, kVec>(p.dx, row * p.ldx, col, p.D, d);
    if (!p.b) continue;
    float rb = 1.f;
    if (p.post != GE_NORM_NONE) rb = normalise(y, p.post, p.eps_post, p.inv_d, p.D, col, row_sum);
    const int64_t g = p.gate && on ? row / p.rows_per_gate : 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if (kWhole) acc_gate[k][i] += d[k][i] * y[k][i];
        else acc_post[k][i] += d[k][i] * y[k][i];
      }
    if (kWhole && on && (row + 1 == end || (row + 1) % p.rows_per_gate == 0)) {
      // the group's last row: its gate's gradient is complete
      float w[NV][kChunk];
      load_w<NV, kVec>(p, p.gate, g * p.D, col, w);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) acc_post[k][i] += w[k][i] * acc_gate[k][i];
      if (p.dgate) {
        load_w<NV, kVec>(p, p.w_post, 0, col, w);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < kChunk; ++i) w[k][i] *= p.alpha * acc_gate[k][i];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (col(k, i) < p.D) putw(p.wt, p.dgate, g * p.D + col(k, i), w[k][i]);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) acc_gate[k][i] = 0.f;
    }
    times_post<NV, kVec>(p, col, own_post, g, at, d);
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
    if (p.db && on) store_row<DT, NV, kVec>(p.db, row * p.ldb, col, p.D, d);
  }
  if (u < p.units) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col(k, i) < p.D) {
          p.part_pre[int64_t(u) * p.D + col(k, i)] = acc_pre[k][i];
          if (p.part_post) p.part_post[int64_t(u) * p.D + col(k, i)] = acc_post[k][i];
        }
  }
}

template <int NV, bool kVec>
const void *pick_run(int dt) {
  return dt == GE_F16    ? reinterpret_cast<const void *>(norm_kernel<GE_F16, NV, kVec>)
         : dt == GE_BF16 ? reinterpret_cast<const void *>(norm_kernel<GE_BF16, NV, kVec>)
                         : reinterpret_cast<const void *>(norm_kernel<GE_F32, NV, kVec>);
}

template <int NV, bool kVec, bool kWhole>
const void *pick_grad(int dt) {
  return dt == GE_F16    ? reinterpret_cast<const void *>(norm_grad_kernel<GE_F16, NV, kVec, kWhole>)
         : dt == GE_BF16 ? reinterpret_cast<const void *>(norm_grad_kernel<GE_BF16, NV, kVec, kWhole>)
                         : reinterpret_cast<const void *>(norm_grad_kernel<GE_F32, NV, kVec, kWhole>);
}

}  // namespace ge
