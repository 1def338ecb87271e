// fp8.cuh -- parameters and handles of the block-scaled 8-bit products.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "xent_math.cuh"

namespace ge {

constexpr int kF8Block = 128;  // columns that share a scale: one k-block, one 128-byte swizzle row

struct Fp8Params {
  CUtensorMap tmA, tmB;    // (K, M), (K, N): boxes of 128 bytes by up to 128 rows
  uint32_t *status;
  uint64_t timeout_ns;
  const float *sa, *sb;    // [k-block][row], [k-block][column or column block]
  int64_t lds_a, lds_b;
  const void *c;           // added, or nullptr
  void *d;
  int64_t ldd;
  int32_t M, N;
  int32_t num_kb, num_m_blk, num_n_blk, raster_group;
  int32_t slices, kb_split;  // a tile's k-blocks are shared by the `slices` CTAs of a cluster, kb_split each
  int32_t stages;
  int32_t a_e5m2, b_e5m2, dt, vec;  // vec: rows of C and D are whole units of 32 bytes (2) or of 16 (1)
  int32_t a_rows;          // rows of an A tile that are loaded (one CTA)
  uint32_t debug_flags;
  uint32_t off_B, off_bar, off_turn;
};

constexpr int kF8Epi0 = 4;                // warps: producer, two MMA, scales, 8 epilogue
constexpr int kF8Threads = 32 * (kF8Epi0 + 8);
// Registers of a thread: all start with 168; the first four warps give some of theirs to the others, whose 128
// sums and 64 values on their way would not fit otherwise.
constexpr int kF8Regs = 168, kF8RegsLess = 72, kF8RegsMore = 216;
static_assert(128 * kF8RegsLess + 256 * kF8RegsMore <= kF8Threads * kF8Regs, "registers to give away");
constexpr uint32_t kF8BarBytes = 256;
// Scales of some k-blocks, two deep: the tile's rows', and its column blocks' or columns'.
__host__ __device__ constexpr int fp8_batch(bool square) { return square ? 8 : 4; }
__host__ __device__ constexpr uint32_t fp8_scale_bytes(int bn, bool square) {
  return 2u * 4u * static_cast<uint32_t>(fp8_batch(square)) * static_cast<uint32_t>(128 + (square ? 2 : bn));
}

// Rows of no whole 16 bytes: an epilogue warp's 32 x 32 sums on their way to D
constexpr int kF8TurnPitch = 33;
constexpr uint32_t kF8TurnBytes = 8u * 32u * kF8TurnPitch * 4u;

constexpr int kF8MaxSlices = 8;
constexpr int kF8PartPitch = 128 + 4;  // floats between the rows of a slice's sums in shared memory

// square: B's scales are one for each 128 columns; add: there is a C; turned: rows of C and D are no whole 16 bytes
const void *fp8_kernel_cg1(bool square, bool add, bool turned);  // 128 x 128 tiles, one CTA
const void *fp8_kernel_cg2(bool square, bool add, bool turned);  // 256 x 256 tiles, a CTA pair


// few rows of A (fp8_few.cu)
constexpr int kF8FewRows = 16, kF8FewUnit = 16;  // rows of A at most, rows of B that a CTA takes at a time
constexpr int kF8FewThreads = 256, kF8FewPerSm = 2;
struct Fp8Few {
  const void *fn;
  int smem;
};
Fp8Few fp8_few(bool a_e5m2, bool b_e5m2, int M);

#ifdef __CUDACC__
__device__ __forceinline__ float load_one(const void *p, int64_t at, int dt) {
  if (dt == GE_F32) return static_cast<const float *>(p)[at];
  const uint16_t v = static_cast<const uint16_t *>(p)[at];
  return dt == GE_BF16 ? __uint_as_float(uint32_t(v) << 16) : __half2float(__ushort_as_half(v));
}

__device__ __forceinline__ void store_one(void *p, int64_t at, int dt, float v) {
  if (dt == GE_F32) static_cast<float *>(p)[at] = v;
  else static_cast<uint16_t *>(p)[at] = static_cast<uint16_t>(pack16(dt == GE_BF16, v, 0.f));
}
#endif

}  // namespace ge
