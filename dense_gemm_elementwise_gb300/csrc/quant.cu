// quant.cu -- 8-bit values and scales for blocks of 128 (gemm_epi_quant_*).
//
//   scale = max(amax / largest q, 2^-126),  q = round(x / scale)
//
// A CTA holds a tile of 128 x 128 elements in registers: a thread has 8 rows of 8
// columns, so that a block of a row lies with 16 lanes (four shuffles for its maximum), a
// thread's own columns give 8 bytes of 8 rows of the transposed matrix, and everything is made
// from one reading of x.  The transposed values cross the CTA through 16 KiB of shared memory,
// whose 8-byte units are permuted so that writes and reads touch every bank equally often.
//
// Bound by memory: x once, one byte per element and output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "gemm_epi.h"
#include "host.h"
#include "ptx.cuh"

using namespace ge;

namespace {

constexpr int kB = 128;           // a block's side
constexpr int kQuantThreads = 256;

struct QuantParams {
  const void *x;
  uint8_t *q, *qt;
  float *scale, *scale_t;
  int64_t ldx, ldq, ldqt, lds, ldst;
  int32_t T, D;
  int32_t e5m2, square;
  float largest;
};

// two values as 8-bit floats, lo in the lower byte
__device__ __forceinline__ uint32_t pack8(bool e5m2, float lo, float hi) {
  uint16_t r;
  if (e5m2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 consecutive elements of a row
template <int XT>
struct Eight {
  uint4 r;
  __device__ __forceinline__ float at(int j) const {
    const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
    if constexpr (XT == GE_BF16) return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(j & 1 ? w >> 16 : w)));
  }
  __device__ __forceinline__ void load(const void *p) { r = __ldg(static_cast<const uint4 *>(p)); }
  // magnitudes' maxima, two at a time; NaN is none
  struct Tops {
    uint32_t w[4];
  };
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t m;
    if constexpr (XT == GE_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
  }
  static __device__ __forceinline__ float wide(uint32_t w, int half) {
    Eight e;
    e.r.x = w;
    return e.at(half);
  }
  // this row's maximum; the columns' so far go into `cols`
  __device__ __forceinline__ float top(Tops &cols) const {
    const uint32_t a[4] = {r.x & 0x7fff7fffu, r.y & 0x7fff7fffu, r.z & 0x7fff7fffu, r.w & 0x7fff7fffu};
#pragma unroll
    for (int j = 0; j < 4; ++j) cols.w[j] = max2(cols.w[j], a[j]);
    const uint32_t m = max2(max2(a[0], a[1]), max2(a[2], a[3]));
    return fmaxf(wide(m, 0), wide(m, 1));
  }
  static __device__ __forceinline__ float at(const Tops &c, int j) { return wide(c.w[j >> 1], j & 1); }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load_some(const void *p, int n) {
    const uint16_t *s = static_cast<const uint16_t *>(p);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (2 * j < n ? __ldg(s + 2 * j) : 0u) | (2 * j + 1 < n ? uint32_t(__ldg(s + 2 * j + 1)) << 16 : 0u);
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Eight<GE_F32> {
  float4 a, b;
  __device__ __forceinline__ float at(int j) const {
    const float4 &v = j < 4 ? a : b;
    return (j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w;
  }
  struct Tops {
    float w[8];
  };
  __device__ __forceinline__ float top(Tops &cols) const {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(at(j));
      m = fmaxf(m, x);
      cols.w[j] = fmaxf(cols.w[j], x);
    }
    return m;
  }
  static __device__ __forceinline__ float at(const Tops &c, int j) { return c.w[j]; }
  __device__ __forceinline__ void load(const void *p) {
    a = __ldg(static_cast<const float4 *>(p));
    b = __ldg(static_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load_some(const void *p, int n) {
    const float *s = static_cast<const float *>(p);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? __ldg(s + j) : 0.f;
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ float scale_of(float amax, float largest) { return fmaxf(__fdiv_rn(amax, largest), 0x1p-126f); }

// 8 bytes, of which n exist
__device__ __forceinline__ void store8(uint8_t *p, uint32_t lo, uint32_t hi, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
  } else {
    for (int j = 0; j < n; ++j) p[j] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
  }
}

// The maxima of 2 N values over the two lanes that differ in bit `o`: each keeps N of them, the upper half where it has the bit.
template <int N>
__device__ __forceinline__ void halve(float (&v)[8], int o) {
  const bool upper = (threadIdx.x & o) != 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float keep = upper ? v[N + i] : v[i], give = upper ? v[i] : v[N + i];
    v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
  }
}

template <int XT, bool COLS>
__global__ void __launch_bounds__(kQuantThreads, XT == GE_F32 ? 2 : 4) quant_kernel(const __grid_constant__ QuantParams p, bool vec) {
  __shared__ __align__(16) float part[8][kB];        // columns' maxima, by warp
  __shared__ __align__(16) float inverse[kB];        // columns' inverse scales
  __shared__ __align__(16) uint8_t turned[COLS ? kB * kB : 16];
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles_d = (p.D - 1) / kB + 1, td = blockIdx.x % tiles_d, tt = blockIdx.x / tiles_d;
  const int64_t d0 = int64_t(td) * kB, t0 = int64_t(tt) * kB;
  const int64_t d = d0 + cg * 8, t = t0 + rg * 8;
  const int cols = static_cast<int>(min(int64_t(8), p.D - d)), rows = static_cast<int>(min(int64_t(8), p.T - t));
  constexpr int es = XT == GE_F32 ? 4 : 2;
  griddep_wait();
  griddep_launch_dependents();
  Eight<XT> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const char *s = static_cast<const char *>(p.x) + ((t + i) * p.ldx + d) * es;
    if (i >= rows || cols <= 0) v[i].zero();
    else if (vec && cols == 8) v[i].load(s);
    else v[i].load_some(s, cols);
  }
  typename Eight<XT>::Tops tops = {};
  float top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = v[i].top(tops);
  // A scale is a division and its inverse another, which take as many instructions as all else that an
  // element needs: each is made by one thread (81 us for 16384 x 4096 both ways, when every thread made its own).
  float row_inv[8], col_inv[8];
  if (p.square) {
    float m = top[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, top[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) part[0][warp] = m;
    __syncthreads();
    m = part[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = fmaxf(m, part[0][w]);
    const float s = scale_of(m, p.largest), inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) row_inv[i] = col_inv[i] = inv;
    if (threadIdx.x == 0) {
      if (p.q) p.scale[td * p.lds + tt] = s;
      if (COLS) p.scale_t[tt * p.ldst + td] = s;
    }
  } else {
    if (COLS) {
      float c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = Eight<XT>::at(tops, j);
      halve<4>(c, 16);
      *reinterpret_cast<float4 *>(&part[warp][cg * 8 + (lane >> 4) * 4]) = make_float4(c[0], c[1], c[2], c[3]);
      __syncthreads();
      if (threadIdx.x < kB) {
        float m = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = fmaxf(m, part[w][threadIdx.x]);
        const float s = scale_of(m, p.largest);
        inverse[threadIdx.x] = __frcp_rn(s);
        if (d0 + threadIdx.x < p.D) p.scale_t[tt * p.ldst + d0 + threadIdx.x] = s;
      }
    }
    if (p.q) {
      // lanes 2i and 2i + 1 of 16 end with row i's maximum
      halve<4>(top, 8);
      halve<2>(top, 4);
      halve<1>(top, 2);
      const float m = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], 1));
      const float s = scale_of(m, p.largest), inv = __frcp_rn(s);
      const int i = cg >> 1;
      if ((cg & 1) == 0 && i < rows) p.scale[td * p.lds + t + i] = s;
#pragma unroll
      for (int k = 0; k < 8; ++k) row_inv[k] = __shfl_sync(0xffffffffu, inv, (lane & 16) | (2 * k));
    }
  }
  if (p.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= rows) break;
      const float r = row_inv[i];
      const uint32_t lo = pack8(p.e5m2, v[i].at(0) * r, v[i].at(1) * r) | pack8(p.e5m2, v[i].at(2) * r, v[i].at(3) * r) << 16;
      const uint32_t hi = pack8(p.e5m2, v[i].at(4) * r, v[i].at(5) * r) | pack8(p.e5m2, v[i].at(6) * r, v[i].at(7) * r) << 16;
      if (cols > 0) store8(p.q + (t + i) * p.ldq + d, lo, hi, cols);
    }
  }
  if constexpr (COLS) {
    if (!p.square) {
      __syncthreads();
      const float4 a = *reinterpret_cast<const float4 *>(&inverse[cg * 8]), b = *reinterpret_cast<const float4 *>(&inverse[cg * 8 + 4]);
      col_inv[0] = a.x, col_inv[1] = a.y, col_inv[2] = a.z, col_inv[3] = a.w;
      col_inv[4] = b.x, col_inv[5] = b.y, col_inv[6] = b.z, col_inv[7] = b.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = col_inv[j];
      const uint32_t lo = pack8(p.e5m2, v[0].at(j) * r, v[1].at(j) * r) | pack8(p.e5m2, v[2].at(j) * r, v[3].at(j) * r) << 16;
      const uint32_t hi = pack8(p.e5m2, v[4].at(j) * r, v[5].at(j) * r) | pack8(p.e5m2, v[6].at(j) * r, v[7].at(j) * r) << 16;
      *reinterpret_cast<uint2 *>(turned + (cg * 8 + j) * kB + ((rg ^ cg) << 3)) = make_uint2(lo, hi);
    }
    __syncthreads();
    // 16 lanes write the 128 bytes of a column
    const int left = static_cast<int>(min(int64_t(8), p.T - (t0 + cg * 8)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = rg + 16 * i;
      if (d0 + c >= p.D || left <= 0) continue;
      const uint2 w = *reinterpret_cast<const uint2 *>(turned + c * kB + ((cg ^ (c >> 3)) << 3));
      store8(p.qt + (d0 + c) * p.ldqt + t0 + cg * 8, w.x, w.y, left);
    }
  }
}

template <int XT>
const void *pick(bool cols) {
  return cols ? reinterpret_cast<const void *>(quant_kernel<XT, true>) : reinterpret_cast<const void *>(quant_kernel<XT, false>);
}

}  // namespace

struct gemm_epi_quant_plan {
  QuantParams p;
  int32_t x;
  bool vec;  // rows of x are whole 16-byte units
};

extern "C" {

int gemm_epi_quant_plan_create(gemm_epi_quant_plan **plan, int64_t T, int64_t D, const ge_quant_desc *desc) {
  if (!plan) return GE_ERR_INVALID;
  *plan = nullptr;
  if (!desc) return GE_ERR_INVALID;
  if ((desc->x != GE_F16 && desc->x != GE_BF16 && desc->x != GE_F32) || (desc->q != GE_E4M3 && desc->q != GE_E5M2))
    return GE_ERR_UNSUPPORTED;
  if ((desc->block != GE_BLOCK_ROW && desc->block != GE_BLOCK_SQUARE) || desc->reserved != 0) return GE_ERR_INVALID;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  if (T <= 0 || D <= 0 || T > kMost || D > kMost) return GE_ERR_SHAPE;
  ge_quant_desc d = *desc;
  const bool square = d.block == GE_BLOCK_SQUARE;
  const struct { int64_t *ld; int64_t least; bool bytes; } pitch[] = {
      {&d.ldx, D, false}, {&d.ldq, D, true}, {&d.ldqt, T, true},
      {&d.lds, square ? ceil_div(T, kB) : T, false}, {&d.ldst, square ? ceil_div(D, kB) : D, false}};
  for (const auto &q : pitch) {
    if (*q.ld == 0) *q.ld = q.least;  // q's and qt's are looked at when they are asked for
    else if (q.bytes && *q.ld % 16 != 0) return GE_ERR_MISALIGNED;
    if (*q.ld < q.least || *q.ld > kMost) return GE_ERR_SHAPE;
  }
  if (ceil_div(T, kB) * ceil_div(D, kB) > kMost) return GE_ERR_SHAPE;  // a CTA each
  int dev = 0, sms = 0, smem = 0;
  const int st = current_device(&dev, &sms, &smem);
  if (st != GE_OK) return st;
  gemm_epi_quant_plan *pl = new (std::nothrow) gemm_epi_quant_plan();
  if (!pl) return GE_ERR_INVALID;
  std::memset(static_cast<void *>(&pl->p), 0, sizeof(pl->p));
  QuantParams &p = pl->p;
  p.ldx = d.ldx;
  p.ldq = d.ldq;
  p.ldqt = d.ldqt;
  p.lds = d.lds;
  p.ldst = d.ldst;
  p.T = static_cast<int32_t>(T);
  p.D = static_cast<int32_t>(D);
  p.e5m2 = d.q == GE_E5M2;
  p.square = square;
  p.largest = p.e5m2 ? 57344.f : 448.f;
  pl->x = d.x;
  pl->vec = d.ldx * (d.x == GE_F32 ? 4 : 2) % 16 == 0;
  *plan = pl;
  return GE_OK;
}

void gemm_epi_quant_plan_destroy(gemm_epi_quant_plan *plan) { delete plan; }

int gemm_epi_quant_run(gemm_epi_quant_plan *pl, const void *x, void *q, float *scale, void *qt, float *scale_t,
                       void *stream) {
  if (!pl) return GE_ERR_INVALID;
  if (!x || (!q && !qt) || (!q) != (!scale) || (!qt) != (!scale_t)) return GE_ERR_MISSING_ARG;
  if ((q && q == qt) || (scale && scale == scale_t)) return GE_ERR_INVALID;
  for (const void *a : {x, static_cast<const void *>(q), static_cast<const void *>(scale),
                        static_cast<const void *>(qt), static_cast<const void *>(scale_t)})
    if (!is_aligned16(a)) return GE_ERR_MISALIGNED;
  if ((q && pl->p.ldq % 16 != 0) || (qt && pl->p.ldqt % 16 != 0)) return GE_ERR_MISALIGNED;
  QuantParams p = pl->p;
  p.x = x;
  p.q = static_cast<uint8_t *>(q);
  p.scale = scale;
  p.qt = static_cast<uint8_t *>(qt);
  p.scale_t = scale_t;
  const void *fn = pl->x == GE_F32 ? pick<GE_F32>(qt) : pl->x == GE_BF16 ? pick<GE_BF16>(qt) : pick<GE_F16>(qt);
  const dim3 grid(static_cast<unsigned>(ceil_div(p.D, kB) * ceil_div(p.T, kB)));
  void *args[] = {&p, &pl->vec};
  return launch_pdl(fn, grid, dim3(kQuantThreads), 0, args, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GE_OK
                                                                                                              : GE_ERR_CUDA;
}

}  // extern "C"
