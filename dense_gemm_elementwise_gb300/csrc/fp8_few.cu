// fp8_few.cu -- the product of 8-bit floats with a scale for each block of 128, for up to 16 rows of A.
//
//   D^T = C^T + sum_j scale_b[j] scale_a[j] (B_j @ A_j^T)
//
// Bound by reading B once, and by a launch's start and end.  The tensor unit of fp8_kernel.cuh wants 128 rows
// of A, its tiles are 128 rows of B on some of the SMs, and its ring, tensor memory and join take time to
// begin.  Here CTAs have 16 rows of B at a time, and all SMs take part:
//   * A CTA's warps share the blocks of 128 columns.  Each copies its own (B's, A's and their scales) to a ring
//     of its own in shared memory (cp.async), so that warps wait for each other once for 16 rows, not at every block, and loads
//     run on into the next 16 rows.  All of an SM's shared memory is on its way at a time.  (With registers in its place
//     loads share the few counters by which a warp waits for them: 42 us for 8 x 40000 x 4096, here 30, 5.5 TB/s.)
//   * B's rows are the 16 rows of mma.sync m16n8k16, A's rows its 8 columns; 8-bit floats are exact in fp16 and
//     products are summed in fp32 over a block, then scaled and added.  (8-bit operands of mma.sync: 2 % slower.)  A lane
//     reads 32 consecutive bytes of a row, whose columns it calls 2q, 2q + 1, 2q + 8, 2q + 9 of a step, on both sides.
//   * The warps' sums are added in order: results repeat bit for bit.
// 1 x 8192 x 4096: 9.3 us from memory and 8.1 from the L2, fp8_kernel.cuh 11.3 and 10.3; 1 x 2048 x 2048 2.9 and 5.9;
// 8 x 2048 x 7168 5.3 and 9.4.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "gemm_epi.h"
#include "ptx.cuh"
#include "xent_math.cuh"

namespace ge {
namespace {

constexpr int kRows = 16, kTile = 8, kWarps = kF8FewThreads / 32;
constexpr int kSpace = 226 * 1024;  // of an SM's shared memory, each CTA's reserve left out

// four 8-bit floats as fp16 (exact)
template <bool E5M2>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint16_t a = static_cast<uint16_t>(w), b = static_cast<uint16_t>(w >> 16);
  if constexpr (E5M2) {
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(lo) : "h"(a));
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(hi) : "h"(b));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(a));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(b));
  }
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3, uint32_t a0, uint32_t a1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(b0), "r"(b1), "r"(b2), "r"(b3), "r"(a0), "r"(a1));
}

// 16 bytes, of which `n` are there and read; zeros behind them
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t *from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t to, const float *from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

// Up to kTokens rows of A.
template <int kTokens>
struct Few {
  static constexpr int kTiles = (kTokens + kTile - 1) / kTile;
  static constexpr int kSlot = (kRows + kTokens) * kF8Block + 128;  // a block of B's rows and of A's, and their scales
  static constexpr int kPart = kTiles * kTile * (kRows + 1);        // a warp's sums
  static constexpr int kParts = kTokens > 8 ? 1 : 2;                // of two units, where blocks leave room for them
  static constexpr int kDepth =  // blocks of a warp under way
      (kSpace / kF8FewPerSm - 128 - 4 * kWarps * kPart * kParts) / (kWarps * kSlot);
  static_assert(kDepth >= 2, "blocks under way");
  static constexpr int kSmem = 128 + 4 * kWarps * kPart * kParts + kWarps * kDepth * kSlot;
};

template <bool A5, bool B5, int kTokens>
__global__ void __launch_bounds__(kF8FewThreads, kF8FewPerSm) fp8_few_kernel(const __grid_constant__ Fp8Params p, const uint8_t *a, const uint8_t *b,
                                                                           int64_t lda, int64_t ldb, int32_t K, bool square) {
  using F = Few<kTokens>;
  constexpr int NT = F::kTiles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  uint8_t *ring = smem + warp * F::kDepth * F::kSlot;
  float(*part)[kWarps][NT * kTile][kRows + 1] = reinterpret_cast<float(*)[kWarps][NT * kTile][kRows + 1]>(smem + kWarps * F::kDepth * F::kSlot);
  griddep_wait();
  griddep_launch_dependents();
  const int units = (p.N + kRows - 1) / kRows;
  // All warps go through as many blocks of each unit, some of which do not exist; loads run on into the next unit.
  const int most = (p.num_kb + kWarps - 1) / kWarps * kWarps;
  int ahead = blockIdx.x, its = warp, to = 0;
  auto fill = [&]() {
    if (ahead < units && its < p.num_kb) {
      // 8 lanes copy a row's 128 bytes, in an order that lets reads touch every bank equally often
      const int r0 = lane >> 3, c = lane & 7, k = its * kF8Block + c * 16, n = max(0, min(16, K - k));
      const uint32_t slot = smem_u32(ring) + to * F::kSlot;
      const int64_t at = n > 0 ? k : 0;
#pragma unroll
      for (int j = 0; j < kRows / 4; ++j) {
        const int r = r0 + 4 * j;  // (a row that does not exist is another's, and left out in the end)
        copy16(slot + r * kF8Block + ((c ^ (r & 7)) << 4), b + min(ahead * kRows + r, p.N - 1) * ldb + at, n);
      }
#pragma unroll
      for (int j = 0; j < (kTokens + 3) / 4; ++j) {
        const int r = r0 + 4 * j;
        if (r < p.M) copy16(slot + (kRows + r) * kF8Block + ((c ^ (r & 7)) << 4), a + r * lda + at, n);
      }
      const uint32_t scale = slot + (kRows + kTokens) * kF8Block + lane * 4;
      if (lane < kRows) copy4(scale, p.sb + int64_t(its) * p.lds_b + (square ? ahead * kRows / kF8Block : min(ahead * kRows + lane, p.N - 1)));
      else if (lane - kRows < p.M) copy4(scale, p.sa + int64_t(its) * p.lds_a + lane - kRows);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    its += kWarps;
    if (its >= most) its = warp, ahead += gridDim.x;
    if (++to == F::kDepth) to = 0;
  };
#pragma unroll 1
  for (int i = 0; i < F::kDepth; ++i) fill();
  int from = 0, turn = 0;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    float acc[NT][4] = {};
#pragma unroll 1
    for (int kb = warp; kb < most; kb += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(F::kDepth - 1) : "memory");
      __syncwarp();
      if (kb < p.num_kb) {
        const uint8_t *slot = ring + from * F::kSlot;
        const float *scale = reinterpret_cast<const float *>(slot + (kRows + kTokens) * kF8Block);
        float d[NT][4] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = ((2 * q + i) ^ g) << 4;
          const uint4 w0 = *reinterpret_cast<const uint4 *>(slot + g * kF8Block + at), w1 = *reinterpret_cast<const uint4 *>(slot + (g + 8) * kF8Block + at);
          uint4 v[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t)  // (what other tokens' places hold stays in their columns)
            v[t] = *reinterpret_cast<const uint4 *>(slot + (kRows + (t * kTile + g) % kTokens) * kF8Block + (((2 * q + i) ^ (((t * kTile + g) % kTokens) & 7)) << 4));
          const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t r0[2], r1[2];
            widen4<B5>(x0[u], r0[0], r0[1]);
            widen4<B5>(x1[u], r1[0], r1[1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t y[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
              uint32_t e[2];
              widen4<A5>(y[u], e[0], e[1]);
              mma(d[t], r0[0], r1[0], r0[1], r1[1], e[0], e[1]);
            }
          }
        }
        const float sb[2] = {scale[g], scale[g + 8]};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float sa = scale[kRows + (t * kTile + 2 * q + (j & 1)) % kTokens];
            acc[t][j] = fmaf(d[t][j] * sb[j >> 1], sa, acc[t][j]);
          }
      }
      if (++from == F::kDepth) from = 0;
      __syncwarp();
      fill();
    }
    // (a buffer's last readers have passed a barrier since)
    float(&sums)[kWarps][NT * kTile][kRows + 1] = part[turn];
    if (F::kParts == 2) turn ^= 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[warp][t * kTile + 2 * q + (j & 1)][g + 8 * (j >> 1)] = acc[t][j];
    __syncthreads();
    for (int i = threadIdx.x; i < min(p.M, kTokens) * kRows; i += kF8FewThreads) {
      const int m = i / kRows, n = unit * kRows + i % kRows;
      if (n >= p.N) continue;
      float v = sums[0][m][i % kRows];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) v += sums[w][m][i % kRows];
      const int64_t at = m * p.ldd + n;
      store_one(p.d, at, p.dt, v + (p.c ? load_one(p.c, at, p.dt) : 0.f));
    }
    if (F::kParts == 1) __syncthreads();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool A5, bool B5, int kTokens>
Fp8Few kernel() {
  return {reinterpret_cast<const void *>(fp8_few_kernel<A5, B5, kTokens>), Few<kTokens>::kSmem};
}

template <bool A5, bool B5>
Fp8Few pick(int M) {
  return M <= 2 ? kernel<A5, B5, 2>() : M <= 8 ? kernel<A5, B5, 8>() : kernel<A5, B5, 16>();
}

}  // namespace

Fp8Few fp8_few(bool a_e5m2, bool b_e5m2, int M) {
  return a_e5m2 ? (b_e5m2 ? pick<true, true>(M) : pick<true, false>(M)) : (b_e5m2 ? pick<false, true>(M) : pick<false, false>(M));
}

}  // namespace ge
