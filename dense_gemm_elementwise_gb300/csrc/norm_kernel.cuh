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

#include <type_traits>

#include "gemm_epi.h"
#include "norm.h"
#include "ptx.cuh"

namespace ge {


template <int DT> struct Elem;
template <> struct Elem<GE_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ float2 get2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
  static __device__ __forceinline__ uint32_t put2(float2 v) {
    const __half2 h = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
};
template <> struct Elem<GE_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ float2 get2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t put2(float2 v) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
};
template <> struct Elem<GE_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};

// Two fp32 operations per instruction: these kernels do about 40 for every
// element of 2 bytes, and the instructions issued were what bound them (0.7
// of the schedulers' slots at 0.6 of the memory's rate).
union Pair { float2 f; unsigned long long u; };
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  Pair x{a}, y{b}, z{c}, r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(x.u), "l"(y.u), "l"(z.u));
  return r.f;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  Pair x{a}, y{b}, r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(x.u), "l"(y.u));
  return r.f;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  Pair x{a}, y{b}, r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(x.u), "l"(y.u));
  return r.f;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

constexpr int kPairs = kChunk / 2;

// How a thread reaches its columns.
//   P_RING     rows of whole 16-byte units: 8 columns in a run, moved 16 bytes at
//              a time, rows on their way in a ring in shared memory
//   P_DIRECT   the same for rows too wide for a ring, read when they are wanted
//              (each thread then has 8 or 16 loads in flight)
//   P_STRIDED  other rows: every row_threads-th column, so that the threads of a
//              warp read neighbouring elements (8 in a run would have each load
//              touch four times the cache lines); fp32 through the ring
//   P_PAIRS    the same, two columns at a time and through the ring, where row
//              pitches are even
enum Path { P_RING = 0, P_DIRECT = 1, P_STRIDED = 2, P_PAIRS = 3 };

template <int PATH>
struct Columns {
  int t, per;
  __device__ __forceinline__ int operator()(int k, int i) const {
    return PATH == P_PAIRS     ? 2 * ((k * kPairs + i / 2) * per + t) + (i & 1)
           : PATH == P_STRIDED ? (k * kChunk + i) * per + t
                               : (t + k * per) * kChunk + i;
  }
};

// row: the row's first element
template <int DT, int NV, int PATH>
__device__ __forceinline__ void store_row(typename Elem<DT>::T *row, const Columns<PATH> &col, int D,
                                          const float2 (&v)[NV][kPairs]) {
  using E = Elem<DT>;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if constexpr (PATH == P_PAIRS) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        if (col(k, 2 * j) >= D) continue;
        if (col(k, 2 * j) + 1 == D) row[D - 1] = E::put(v[k][j].x);  // an odd row's last
        else if constexpr (DT == GE_F32) *reinterpret_cast<float2 *>(row + col(k, 2 * j)) = v[k][j];
        else *reinterpret_cast<uint32_t *>(row + col(k, 2 * j)) = E::put2(v[k][j]);
      }
    } else if (PATH < P_STRIDED && col(k, 0) + kChunk <= D) {
      uint4 *q = reinterpret_cast<uint4 *>(row + col(k, 0));
      if constexpr (DT == GE_F32) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          q[j] = make_uint4(__float_as_uint(v[k][2 * j].x), __float_as_uint(v[k][2 * j].y),
                            __float_as_uint(v[k][2 * j + 1].x), __float_as_uint(v[k][2 * j + 1].y));
      } else {
        *q = make_uint4(E::put2(v[k][0]), E::put2(v[k][1]), E::put2(v[k][2]), E::put2(v[k][3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col(k, i) < D) row[col(k, i)] = E::put(i & 1 ? v[k][i / 2].y : v[k][i / 2].x);
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

// Factors of a thread's columns, kept in fp32 in shared memory of its own:
// `threads` 16-byte words side by side, so that a warp's accesses are free of
// conflicts, and no barrier: nobody else reads them.
struct Own {
  float4 *base;   // this thread's first word
  int threads;
  template <int NV>
  __device__ __forceinline__ void put(const float2 (&w)[NV][kPairs]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        base[(2 * k + j) * threads] = make_float4(w[k][2 * j].x, w[k][2 * j].y, w[k][2 * j + 1].x, w[k][2 * j + 1].y);
  }
  template <int NV>
  __device__ __forceinline__ void get(float2 (&w)[NV][kPairs]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 f = base[(2 * k + j) * threads];
        w[k][2 * j] = make_float2(f.x, f.y);
        w[k][2 * j + 1] = make_float2(f.z, f.w);
      }
  }
  template <int NV>
  __device__ __forceinline__ void times(float2 (&v)[NV][kPairs]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 f = base[(2 * k + j) * threads];
        v[k][2 * j] = mul2(v[k][2 * j], make_float2(f.x, f.y));
        v[k][2 * j + 1] = mul2(v[k][2 * j + 1], make_float2(f.z, f.w));
      }
  }
  // scale * a[off + column] * b[column], 0 past the end; a vector that is NULL
  // counts as 1.  Not inlined: it runs once for many rows, and its
  // instructions would crowd out the others'; one chunk at a time, to leave the
  // callers their registers.
  template <int NV, int PATH>
  __device__ __noinline__ void fill(const NormParams &p, const Columns<PATH> &col, float scale, const void *a,
                                    int64_t off, const void *b) const {
    if (PATH < P_STRIDED && NV <= 2 && p.w_vec && p.wt != GE_F32 && a) {
      // every load is on its way before the first is used (8192 x 4096 bf16: 46.7 -> 45.0 us, with a
      // gate for every row 82 -> 73)
      uint4 x[NV], y[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        x[k] = y[k] = make_uint4(0, 0, 0, 0);
        if (col(k, 0) >= p.D) continue;
        x[k] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a) + off + col(k, 0));
        if (b) y[k] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(b) + col(k, 0));
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float2 f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u = j ? (i ? x[k].w : x[k].z) : (i ? x[k].y : x[k].x);
            const uint32_t v = j ? (i ? y[k].w : y[k].z) : (i ? y[k].y : y[k].x);
            f[i] = mul2(p.wt == GE_F16 ? Elem<GE_F16>::get2(u) : Elem<GE_BF16>::get2(u), both(scale));
            if (b) f[i] = mul2(f[i], p.wt == GE_F16 ? Elem<GE_F16>::get2(v) : Elem<GE_BF16>::get2(v));
          }
          base[(2 * k + j) * threads] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        }
      return;
    }
#pragma unroll 1
    for (int k = 0; k < NV; ++k) {
      // the loads of both vectors are on their way before the first is used
      float f[kChunk], g[kChunk];
      if (p.wt == GE_F32) read<GE_F32>(p, col, k, a, off, f), read<GE_F32>(p, col, k, b, 0, g);
      else if (p.wt == GE_F16) read<GE_F16>(p, col, k, a, off, f), read<GE_F16>(p, col, k, b, 0, g);
      else read<GE_BF16>(p, col, k, a, off, f), read<GE_BF16>(p, col, k, b, 0, g);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) f[i] *= g[i];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) f[i] = col(k, i) < p.D ? scale * f[i] : 0.f;
      base[2 * k * threads] = make_float4(f[0], f[1], f[2], f[3]);
      base[(2 * k + 1) * threads] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  template <int WT, int PATH>
  static __device__ __forceinline__ void read(const NormParams &p, const Columns<PATH> &col, int k, const void *v,
                                              int64_t off, float (&f)[kChunk]) {
    using T = typename Elem<WT>::T;
    const T *q = static_cast<const T *>(v) + off;
    if (!v) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) f[i] = 1.f;
    } else if (PATH < P_STRIDED && WT != GE_F32 && p.w_vec && col(k, 0) < p.D) {
      union { uint4 w; T e[kChunk]; } u;
      u.w = *reinterpret_cast<const uint4 *>(q + col(k, 0));
#pragma unroll
      for (int i = 0; i < kChunk; ++i) f[i] = Elem<WT>::get(u.e[i]);
    } else if (PATH < P_STRIDED && WT == GE_F32 && p.w_vec) {
      // halves that do not exist: the last that does, dropped by the caller
      const float4 lo = *reinterpret_cast<const float4 *>(q + min(col(k, 0), p.D - 4)),
                   hi = *reinterpret_cast<const float4 *>(q + min(col(k, 4), p.D - 4));
      f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
      f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) f[i] = Elem<WT>::get(q[min(col(k, i), p.D - 1)]);
    }
  }
  // what is kept, to a row of the weights' type
  template <int NV, int PATH>
  __device__ __noinline__ void store(const NormParams &p, const Columns<PATH> &col, void *out, int64_t off) const {
#pragma unroll 1
    for (int k = 0; k < NV; ++k) {
      const float4 lo = base[2 * k * threads], hi = base[(2 * k + 1) * threads];
      const float f[kChunk] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      if (PATH < P_STRIDED && p.w_vec) {  // 16 bytes at a time: of fp32 two halves, of which one may exist
        if (p.wt == GE_F32) {
          float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(out) + off + col(k, 0));
          if (col(k, 0) < p.D) q[0] = lo;
          if (col(k, 4) < p.D) q[1] = hi;
        } else if (col(k, 0) < p.D) {
          uint32_t w[kPairs];
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const float2 v = make_float2(f[2 * j], f[2 * j + 1]);
            w[j] = p.wt == GE_F16 ? Elem<GE_F16>::put2(v) : Elem<GE_BF16>::put2(v);
          }
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + off + col(k, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col(k, i) < p.D) putw(p.wt, out, off + col(k, i), f[i]);
    }
  }
  // Asks for what the next fill from a[off] will read (of the next gate group while this one's
  // rows are worked on: with a gate for every row, 8192 x 4096 bf16, 82 us instead of 91).
  template <int NV, int PATH>
  static __device__ __forceinline__ void prefetch(const NormParams &p, const Columns<PATH> &col, const void *a, int64_t off) {
    if (PATH >= P_STRIDED) return;
#pragma unroll 1
    for (int k = 0; k < NV; ++k)
      if (col(k, 0) < p.D)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t *>(a) + (off + col(k, 0)) * (p.wt == GE_F32 ? 4 : 2)));
  }
};

// Whether rows come through a ring in shared memory: copies of 16 bytes, or of one
// or two elements of 4 or 8 bytes in all (with two columns per load into registers instead,
// 13390 x 4594 bf16 took 268 us and its gradients 514, against 179 and 440).
// kBound: threads that the registers must suffice for; 1024 threads' rows do not
// fit in shared memory.
template <int DT, int PATH, int kBound>
constexpr bool kBySmall = (PATH == P_PAIRS || (PATH == P_STRIDED && DT == GE_F32)) && kBound < kMaxThreads;
template <int DT, int PATH, int kBound>
constexpr bool kByRing = PATH == P_RING || kBySmall<DT, PATH, kBound>;

// Rows on their way from memory: NA tensors of them, `ahead` rows by cp.async
// into the thread's own words of shared memory.  Odd rows of 16-bit elements, which
// cp.async cannot move: the next row's elements in registers, asked for once
// the current row's have been taken. CTAs of over 512 threads have neither room nor
// registers and read a row when it is wanted.
template <int DT, int NV, int PATH, int NA, int kBound>
struct Ring {
  using T = typename Elem<DT>::T;
  static constexpr int kWords = kChunk * sizeof(T) / 16;  // of one tensor's chunk
  static constexpr int kRow = NA * NV * kWords;           // 16-byte words of a thread per row
  static constexpr bool kSmall = kBySmall<DT, PATH, kBound>;
  static constexpr int kUnits = PATH == P_PAIRS ? kPairs : kChunk;  // of a chunk, one copy each
  static constexpr int kUnit = kChunk / kUnits * sizeof(T);         // bytes of one
  uint4 *base;
  int threads, ahead, D;
  Columns<PATH> col;
  static constexpr bool kRaw = PATH == P_STRIDED && kBound <= kVecThreads && !kSmall;
  T raw[kRaw ? NA : 1][kRaw ? NV : 1][kChunk];

  __device__ __forceinline__ Ring(uint4 *base_, int threads_, int ahead_, int D_, const Columns<PATH> &col_)
      : base(base_), threads(threads_), ahead(ahead_), D(D_), col(col_) {}

  // unit u of this thread (small copies); `base` is its first 16-byte word
  __device__ __forceinline__ uint8_t *unit(int u) const {
    return reinterpret_cast<uint8_t *>(base - threadIdx.x) + (u * threads + static_cast<int>(threadIdx.x)) * kUnit;
  }
  // row: the row's first element
  __device__ __forceinline__ void issue(int slot, int a, const T *row) {
    if constexpr (kSmall) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
          const uint32_t dst = smem_u32(unit(((slot * NA + a) * NV + k) * kUnits + j));
          // past the end: the row's last column or pair, dropped when it is taken
          if constexpr (PATH == P_PAIRS) {
            // of an odd row's last pair only what exists is read
            const int c = min(col(k, 2 * j), (D - 1) & ~1), left = c + 1 == D ? kUnit / 2 : kUnit;
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(row + c), "n"(kUnit), "r"(left)
                         : "memory");
          } else {
            const int c = min(col(k, j), D - 1);
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(row + c), "n"(kUnit) : "memory");
          }
        }
    } else if constexpr (PATH == P_RING) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          constexpr int kPer = 16 / sizeof(T);
          const int c = col(k, 0) + j * kPer;
          // columns past the end arrive as zeros
          const int left = min(max(D - c, 0), kPer) * static_cast<int>(sizeof(T));
          const uint32_t dst = smem_u32(base + (slot * kRow + (a * NV + k) * kWords + j) * threads);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(left > 0 ? row + c : row),
                       "r"(left)
                       : "memory");
        }
    } else if constexpr (kRaw) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) take(row, k, i, raw[a][k]);
    }
  }
  // element i of chunk k, or its pair i, from a row at least D long
  __device__ __forceinline__ void take(const T *row, int k, int i, T (&e)[kChunk]) const {
    if constexpr (PATH == P_PAIRS) {
      using Two = typename std::conditional<sizeof(T) == 4, uint2, uint32_t>::type;
      union { Two w; T e[2]; } u;
      const int c = min(col(k, 2 * i), (D - 1) & ~1);
      if (c + 1 == D) u.e[0] = u.e[1] = row[c];
      else u.w = *reinterpret_cast<const Two *>(row + c);
      e[2 * i] = u.e[0];
      e[2 * i + 1] = u.e[1];
    } else {
      e[i] = row[min(col(k, i), D - 1)];
    }
  }
  __device__ __forceinline__ void commit() const {
    if constexpr (kByRing<DT, PATH, kBound>) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the oldest row of the ring has landed
  __device__ __forceinline__ void wait() const {
    if constexpr (kByRing<DT, PATH, kBound>) {
      if (ahead == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (ahead == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  }
  static __device__ __forceinline__ void widen(const uint4 (&w)[kWords], float2 (&v)[kPairs]) {
    if constexpr (DT == GE_F32) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[2 * j] = make_float2(__uint_as_float(w[j % kWords].x), __uint_as_float(w[j % kWords].y));
        v[2 * j + 1] = make_float2(__uint_as_float(w[j % kWords].z), __uint_as_float(w[j % kWords].w));
      }
    } else {
      v[0] = Elem<DT>::get2(w[0].x);
      v[1] = Elem<DT>::get2(w[0].y);
      v[2] = Elem<DT>::get2(w[0].z);
      v[3] = Elem<DT>::get2(w[0].w);
    }
  }
  // row, on: where a row that is read now is, and whether it is there (else `row` is some row that is)
  __device__ __forceinline__ void get(int slot, int a, const T *row, bool on, float2 (&v)[NV][kPairs]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (PATH == P_RING) {
        uint4 w[kWords];
#pragma unroll
        for (int j = 0; j < kWords; ++j) w[j] = base[(slot * kRow + (a * NV + k) * kWords + j) * threads];
        widen(w, v[k]);
      } else if constexpr (PATH == P_DIRECT) {
        if (on && col(k, 0) + kChunk <= D) {
          uint4 w[kWords];
#pragma unroll
          for (int j = 0; j < kWords; ++j) w[j] = reinterpret_cast<const uint4 *>(row + col(k, 0))[j];
          widen(w, v[k]);
        } else {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            v[k][i].x = on && col(k, 2 * i) < D ? Elem<DT>::get(row[col(k, 2 * i)]) : 0.f;
            v[k][i].y = on && col(k, 2 * i + 1) < D ? Elem<DT>::get(row[col(k, 2 * i + 1)]) : 0.f;
          }
        }
      } else {
        T e[kChunk];
        if constexpr (kSmall) {
#pragma unroll
          for (int j = 0; j < kUnits; ++j) {
            using Word = typename std::conditional<kUnit == 8, uint2, uint32_t>::type;
            union { Word w; T e[kChunk / kUnits]; } u;
            u.w = *reinterpret_cast<const Word *>(unit(((slot * NA + a) * NV + k) * kUnits + j));
#pragma unroll
            for (int i = 0; i < kChunk / kUnits; ++i) e[j * (kChunk / kUnits) + i] = u.e[i];
          }
        } else if constexpr (kRaw) {
#pragma unroll
          for (int i = 0; i < kChunk; ++i) e[i] = raw[a][k][i];
        } else {
#pragma unroll
          for (int i = 0; i < (PATH == P_PAIRS ? kPairs : kChunk); ++i) take(row, k, i, e);
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          v[k][i].x = col(k, 2 * i) < D ? Elem<DT>::get(e[2 * i]) : 0.f;
          v[k][i].y = col(k, 2 * i + 1) < D ? Elem<DT>::get(e[2 * i + 1]) : 0.f;
        }
      }
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
    static_assert(K >= 1 && K <= 3, "one to three sums");
    if (per >= 32) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
    } else {
#pragma unroll 1
      for (int s = per >> 1; s > 0; s >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
    }
    if (warps <= 1) return;
    float4 *b = buf + turn;
    turn ^= warps;  // 0 or the second half
    if (lane == 0) b[warp] = make_float4(v[0], v[K > 1 ? 1 : 0], v[K > 2 ? 2 : 0], 0.f);
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(per) : "memory");
    // every warp adds the warps' sums, up to 32 of them, in the same order
    const float4 f = lane < warps ? b[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = f.x;
    if constexpr (K > 1) v[1] = f.y;
    if constexpr (K > 2) v[2] = f.z;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      if (s < warps)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
    // with up to 16 warps the first lane holds the whole sum
    if (warps <= 16)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
  }
};

template <int NV>
__device__ __forceinline__ float sum_of(const float2 (&v)[NV][kPairs]) {
  float2 s = both(0.f);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) s = add2(s, v[k][i]);
  return s.x + s.y;
}

template <int NV>
__device__ __forceinline__ float dot_of(const float2 (&a)[NV][kPairs], const float2 (&b)[NV][kPairs]) {
  float2 s = both(0.f);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) s = fma2(a[k][i], b[k][i], s);
  return s.x + s.y;
}

// v -= mean; columns past the end are 0 and stay 0
template <int NV, int PATH>
__device__ __forceinline__ void centre(float2 (&v)[NV][kPairs], float mean, int D, const Columns<PATH> &col) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      v[k][i].x = col(k, 2 * i) < D ? v[k][i].x - mean : 0.f;
      v[k][i].y = col(k, 2 * i + 1) < D ? v[k][i].y - mean : 0.f;
    }
}

// The inverse divisor of a row; a centred row (GE_NORM_LAYER) has its mean taken off v.
template <int NV, int PATH>
__device__ __forceinline__ float divisor(float2 (&v)[NV][kPairs], int kind, float eps, float inv_d, int D,
                                         const Columns<PATH> &col, RowSum &row_sum) {
  if (kind == GE_NORM_LAYER) {
    float m[1] = {sum_of(v)};
    row_sum(m);
    centre(v, m[0] * inv_d, D, col);
  }
  float s[1] = {dot_of(v, v)};
  row_sum(s);
  return rsqrtf(s[0] * inv_d + eps);
}

// A thread's row and place in it.  Shared memory of a CTA: the rows' sums, then the
// factors w_pre and alpha gate w_post of each thread's columns, then the ring.
template <int PATH>
struct Place {
  int per, mine, t;
  __device__ __forceinline__ Place(int row_threads)
      : per(row_threads), mine(threadIdx.x / row_threads), t(threadIdx.x - mine * row_threads) {}
  __device__ __forceinline__ Columns<PATH> columns() const { return Columns<PATH>{t, per}; }
  __device__ __forceinline__ RowSum row_sum(uint8_t *smem) const {
    const int warps = per / 32;
    return RowSum{reinterpret_cast<float4 *>(smem) + 2 * mine * warps, per, warps, t >> 5,
                  static_cast<int>(threadIdx.x & 31), 1 + mine, 0};
  }
};

// The gate group of a row: divided out only where the last one's rows end.
struct Group {
  int32_t size, g, begin;
  __device__ __forceinline__ void move(int32_t row) {
    if (static_cast<uint32_t>(row - begin) >= static_cast<uint32_t>(size)) {
      g = row / size;
      begin = g * size;
    }
  }
  __device__ __forceinline__ bool last(int32_t row) const { return row - begin == size - 1; }
};

// kBound: threads that the registers must suffice for
template <int DT, int NV, int PATH, int kBound>
__global__ void __launch_bounds__(kBound, 1) norm_kernel(const __grid_constant__ NormParams p) {
  using T = typename Elem<DT>::T;
  constexpr bool kAsk = kByRing<DT, PATH, kBound>;  // rows are asked for ahead of the one at hand
  extern __shared__ __align__(16) uint8_t smem[];
  const Place<PATH> pl(p.row_threads);
  const int rows = blockDim.x / pl.per;
  const Columns<PATH> col = pl.columns();
  RowSum row_sum = pl.row_sum(smem);
  float4 *words = reinterpret_cast<float4 *>(smem + kSumBytes) + threadIdx.x;
  const int n = blockDim.x;
  // w_pre; alpha gate w_post of the gate group at hand
  const Own own_pre{words, n}, own_post{words + 2 * NV * n, n};
  Ring<DT, NV, PATH, 2, kBound> ring(reinterpret_cast<uint4 *>(words + 4 * NV * n), n, p.ahead, p.D, col);
  // Rows are dealt out in turn (8192 x 4096 bf16 45.0 us, in runs 47.1), but with gate
  // groups a CTA takes a run of rows, which meets few of them (groups of 12, 15735 x 1808 f16: 49 us,
  // in turn 84).  Every thread's loop is as long.
  const int step = p.rows_per_unit ? rows : gridDim.x * rows;
  int64_t first = int64_t(blockIdx.x) * (p.rows_per_unit ? p.rows_per_unit : rows);
  const int64_t stop = p.rows_per_unit ? min(first + p.rows_per_unit, int64_t(p.T)) : p.T;
  int64_t row = first + pl.mine;
  const T *x = static_cast<const T *>(p.x), *b = static_cast<const T *>(p.b);
  T *y = static_cast<T *>(p.y), *h = static_cast<T *>(p.h);
  griddep_wait();
  griddep_launch_dependents();
  int64_t ahead = row;  // the next row to ask for
  auto fetch = [&](int slot) {
    if (ahead < stop) {
      ring.issue(slot, 0, x + ahead * p.ldx);
      if (b) ring.issue(slot, 1, b + ahead * p.ldb);
    }
    ring.commit();
    ahead += step;
  };
  for (int s = 0; s < (kAsk ? p.ahead - 1 : 1); ++s) fetch(s);
  if (p.w_pre) own_pre.fill<NV>(p, col, 1.f, p.w_pre, 0, nullptr);
  int32_t at = -1;  // the group that own_post is for
  Group group{static_cast<int32_t>(p.rows_per_gate), 0, 0};
  int slot = 0, next = p.ahead - 1;
  for (; first < stop; first += step, row += step) {
    const bool on = row < stop;
    if (kAsk) fetch(next);
    if (++next == p.ahead) next = 0;
    // the factors of the row's gate group: while the row is on its way, but not while it is in
    // registers, which the call would have to save
    auto factors = [&]() {
      if (p.gate && on) group.move(static_cast<int32_t>(row));
      if (at != group.g) {
        at = group.g;
        own_post.fill<NV>(p, col, p.alpha, p.gate, int64_t(at) * p.D, p.w_post);
        if (p.gate && group.begin < p.T - group.size) Own::prefetch<NV>(p, col, p.gate, (int64_t(at) + 1) * p.D);
      }
    };
    if ((PATH < P_STRIDED || kAsk) && b) factors();
    ring.wait();
    float2 v[NV][kPairs];
    if (!kAsk || !b) ring.get(slot, 0, x + (on ? row : 0) * p.ldx, on, v);
    if (b) {
      float2 u[NV][kPairs];
      ring.get(slot, 1, b + (on ? row : 0) * p.ldb, on, u);
      if (!kAsk) fetch(0);
      if (PATH >= P_STRIDED && !kAsk) factors();
      const float r = p.post != GE_NORM_NONE
                          ? divisor(u, p.post, p.eps_post, p.inv_d, p.D, col, row_sum) : 1.f;
      own_post.times(u);
      if (kAsk) ring.get(slot, 0, x + (on ? row : 0) * p.ldx, on, v);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[k][i] = fma2(u[k][i], both(r), v[k][i]);
    } else if (!kAsk) {
      fetch(0);
    }
    if (++slot == p.ahead) slot = 0;
    if (y && on) store_row<DT, NV, PATH>(y + row * p.ldy, col, p.D, v);
    if (h) {
      const float r = divisor(v, p.pre, p.eps_pre, p.inv_d, p.D, col, row_sum);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[k][i] = mul2(v[k][i], both(r));
      if (p.w_pre) own_pre.times(v);
      if (on) store_row<DT, NV, PATH>(h + row * p.ldh, col, p.D, v);
    }
  }
}

// The rows of lane `lane` of unit u: a unit is a CTA, its lanes take runs of rows_per_lane rows.
__device__ __forceinline__ void unit_rows(const NormParams &p, int u, int lane, int64_t &begin, int64_t &end) {
  int64_t stop;
  if (p.units_per_group) {
    const int64_t g = u / p.units_per_group, s = u - g * p.units_per_group;
    begin = g * p.rows_per_gate + s * p.rows_per_unit;
    stop = min(min(begin + p.rows_per_unit, (g + 1) * p.rows_per_gate), int64_t(p.T));
  } else {
    begin = int64_t(u) * p.rows_per_unit;
    stop = min(begin + p.rows_per_unit, int64_t(p.T));
  }
  begin += int64_t(lane) * p.rows_per_lane;
  end = min(begin + p.rows_per_lane, stop);
  begin = min(begin, end);
}

// kWhole: a unit holds whole gate groups
template <int DT, int NV, int PATH, int kBound, bool kWhole>
__global__ void __launch_bounds__(kBound, 1) norm_grad_kernel(const __grid_constant__ NormParams p) {
  using T = typename Elem<DT>::T;
  constexpr bool kAsk = kByRing<DT, PATH, kBound>;
  extern __shared__ __align__(16) uint8_t smem[];
  const Place<PATH> pl(p.row_threads);
  const Columns<PATH> col = pl.columns();
  RowSum row_sum = pl.row_sum(smem);
  float4 *words = reinterpret_cast<float4 *>(smem + kSumBytes) + threadIdx.x;
  const int n = blockDim.x;
  // w_pre; alpha gate w_post of the gate group at hand, or (kWhole) its gate and alpha w_post apart
  constexpr int kFactors = kWhole ? 3 : 2;
  const Own own_pre{words, n}, own_post{words + 2 * NV * n, n}, own_w{words + 4 * NV * n, n};
  Ring<DT, NV, PATH, 4, kBound> ring(
      reinterpret_cast<uint4 *>(words + kFactors * 2 * NV * n), n, p.ahead, p.D, col);
  int64_t row, end;
  unit_rows(p, blockIdx.x, pl.mine, row, end);
  const T *yin = static_cast<const T *>(p.yin), *dh = static_cast<const T *>(p.dh),
          *dy = static_cast<const T *>(p.dy), *b = static_cast<const T *>(p.b);
  T *dx = static_cast<T *>(p.dx), *db = static_cast<T *>(p.db);
  griddep_wait();
  griddep_launch_dependents();
  int64_t ahead = row;  // the next row to ask for
  auto fetch = [&](int slot) {
    if (ahead < end) {
      ring.issue(slot, 0, yin + ahead * p.ldy);
      ring.issue(slot, 1, dh + ahead * p.ldh);
      if (dy) ring.issue(slot, 2, dy + ahead * p.ldy);
      if (b) ring.issue(slot, 3, b + ahead * p.ldb);
    }
    ring.commit();
    ++ahead;
  };
  for (int s = 0; s < (kAsk ? p.ahead - 1 : 1); ++s) fetch(s);
  if (p.w_pre) own_pre.fill<NV>(p, col, 1.f, p.w_pre, 0, nullptr);
  if (kWhole && b) own_w.fill<NV>(p, col, p.alpha, p.w_post, 0, nullptr);
  float2 acc_pre[NV][kPairs], acc_post[NV][kPairs];
  float2 acc_gate[kWhole ? NV : 1][kPairs];  // whole groups: the current group's q
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      acc_pre[k][i] = acc_post[k][i] = both(0.f);
      if (kWhole) acc_gate[k][i] = both(0.f);
    }
  int32_t at = -1;  // the group that own_post is for
  Group group{static_cast<int32_t>(p.rows_per_gate), 0, 0};
  int slot = 0, next = p.ahead - 1;
  const bool layer_b = b && p.post == GE_NORM_LAYER, norm_b = b && p.post != GE_NORM_NONE;
  // every thread goes round as often: row sums hold barriers.  Past a unit's
  // last row what is computed is dropped.
  for (int r = 0; r < p.rows_per_lane; ++r, ++row) {
    const bool on = row < end;
    if (kAsk) fetch(next);
    if (++next == p.ahead) next = 0;
    auto factors = [&]() {  // of the row's gate group, as in the forward pass
      if (p.gate && on) group.move(static_cast<int32_t>(row));
      if (at != group.g) {
        at = group.g;
        own_post.fill<NV>(p, col, kWhole ? 1.f : p.alpha, p.gate, int64_t(at) * p.D, kWhole ? nullptr : p.w_post);
        if (p.gate && group.begin < p.T - group.size) Own::prefetch<NV>(p, col, p.gate, (int64_t(at) + 1) * p.D);
      }
    };
    if ((PATH < P_STRIDED || kAsk) && b) factors();
    ring.wait();
    // y becomes what N_pre divides, d = dh w_pre, q = dh y
    float2 y[NV][kPairs], d[NV][kPairs], q[NV][kPairs];
    ring.get(slot, 0, yin + (on ? row : 0) * p.ldy, on, y);
    ring.get(slot, 1, dh + (on ? row : 0) * p.ldh, on, d);
    float mean_d = 0.f;
    if (p.pre == GE_NORM_LAYER) {
      float s[2];
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) q[k][i] = d[k][i];
      if (p.w_pre) own_pre.times(q);
      s[0] = sum_of(y);
      s[1] = sum_of(q);
      row_sum(s);
      centre(y, s[0] * p.inv_d, p.D, col);
      mean_d = s[1] * p.inv_d;
    }
    float s[2] = {dot_of(y, y), 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) q[k][i] = mul2(d[k][i], y[k][i]);
    if (p.w_pre) {
      float2 sum = both(0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 f = own_pre.base[(2 * k + j) * n];
          const float2 lo = make_float2(f.x, f.y), hi = make_float2(f.z, f.w);
          sum = fma2(q[k][2 * j], lo, sum);
          sum = fma2(q[k][2 * j + 1], hi, sum);
          d[k][2 * j] = mul2(d[k][2 * j], lo);
          d[k][2 * j + 1] = mul2(d[k][2 * j + 1], hi);
        }
      s[1] = sum.x + sum.y;
    } else {
      s[1] = sum_of(q);
    }
    row_sum(s);
    const float ry = rsqrtf(s[0] * p.inv_d + p.eps_pre);
    const float along = -ry * (ry * s[1] * p.inv_d * ry), mean = -ry * mean_d;
    if (on)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) acc_pre[k][i] = fma2(q[k][i], both(ry), acc_pre[k][i]);
    // d becomes the whole gradient of y (past the end of a centred row it is
    // not 0, but the factors it meets there are)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        d[k][i] = fma2(d[k][i], both(ry), fma2(y[k][i], both(along), both(mean)));
    if (dy) {
      ring.get(slot, 2, dy + (on ? row : 0) * p.ldy, on, y);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) d[k][i] = add2(d[k][i], y[k][i]);
    }
    if (b) ring.get(slot, 3, b + (on ? row : 0) * p.ldb, on, y);  // read before dx is written: it may be in b's place
    if (++slot == p.ahead) slot = 0;
    if (!kAsk) fetch(0);
    if (on) store_row<DT, NV, PATH>(dx + row * p.ldx, col, p.D, d);
    if (!b) continue;
    // y is now b, or what N_post divides
    if (PATH >= P_STRIDED && !kAsk) factors();
    if (layer_b) {
      float m[1] = {sum_of(y)};
      row_sum(m);
      centre(y, m[0] * p.inv_d, p.D, col);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) q[k][i] = mul2(d[k][i], y[k][i]);
    own_post.times(d);
    if (kWhole) own_w.times(d);
    float rb = 1.f;
    if (norm_b) {
      float s2[3] = {dot_of(y, y), dot_of(d, y), layer_b ? sum_of(d) : 0.f};
      row_sum(s2);
      rb = rsqrtf(s2[0] * p.inv_d + p.eps_post);
      const float along2 = -rb * (rb * s2[1] * p.inv_d * rb), mean2 = -rb * s2[2] * p.inv_d;
      if (db && on) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < kPairs; ++i)
            d[k][i] = fma2(d[k][i], both(rb), fma2(y[k][i], both(along2), both(mean2)));
      }
    }
    if (db && on) store_row<DT, NV, PATH>(db + row * p.ldb, col, p.D, d);
    if (on)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if (kWhole) acc_gate[k][i] = fma2(q[k][i], both(rb), acc_gate[k][i]);
          else acc_post[k][i] = fma2(q[k][i], both(rb), acc_post[k][i]);
        }
    if (kWhole && on && (row + 1 == end || group.last(static_cast<int32_t>(row)))) {
      // the group's last row: its gate's gradient is complete
      own_post.get(y);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) acc_post[k][i] = fma2(y[k][i], acc_gate[k][i], acc_post[k][i]);
      if (p.dgate) {
        own_w.times(acc_gate);
        own_post.put(acc_gate);  // the next group's gate takes this place
        own_post.store<NV>(p, col, p.dgate, int64_t(group.g) * p.D);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) acc_gate[k][i] = both(0.f);
    }
  }
  // the lanes' sums in order, through the words that held w_pre's factors
  const int lanes = n / pl.per;
  auto over_lanes = [&](float2 (&v)[NV][kPairs]) {
    if (lanes == 1) return;
    own_pre.put(v);
    __syncthreads();
    if (pl.mine == 0)
      for (int l = 1; l < lanes; ++l) {
        float2 w[NV][kPairs];
        Own{own_pre.base + l * pl.per, n}.get(w);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < kPairs; ++i) v[k][i] = add2(v[k][i], w[k][i]);
      }
    __syncthreads();
  };
  if (lanes > 1) __syncthreads();
  over_lanes(acc_pre);
  if (p.part_post) over_lanes(acc_post);
  if (pl.mine == 0) {
    store_row<GE_F32, NV, PATH>(p.part_pre + int64_t(blockIdx.x) * p.ld_part, col, p.D, acc_pre);
    if (p.part_post) store_row<GE_F32, NV, PATH>(p.part_post + int64_t(blockIdx.x) * p.ld_part, col, p.D, acc_post);
  }
}

template <int DT, int NV, int PATH, int kBound>
const void *run_of() {
  return reinterpret_cast<const void *>(norm_kernel<DT, NV, PATH, kBound>);
}

template <int NV, int PATH, int kBound>
const void *pick_run(int dt) {
  return dt == GE_F16    ? run_of<GE_F16, NV, PATH, kBound>()
         : dt == GE_BF16 ? run_of<GE_BF16, NV, PATH, kBound>()
                         : run_of<GE_F32, NV, PATH, kBound>();
}

template <int DT, int NV, int PATH, int kBound, bool kWhole>
const void *grad_of() {
  return reinterpret_cast<const void *>(norm_grad_kernel<DT, NV, PATH, kBound, kWhole>);
}

template <int NV, int PATH, int kBound, bool kWhole>
const void *pick_grad(int dt) {
  return dt == GE_F16    ? grad_of<GE_F16, NV, PATH, kBound, kWhole>()
         : dt == GE_BF16 ? grad_of<GE_BF16, NV, PATH, kBound, kWhole>()
                         : grad_of<GE_F32, NV, PATH, kBound, kWhole>();
}

}  // namespace ge
