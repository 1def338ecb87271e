// fp8.cuh -- parameters and handles of the block-scaled 8-bit products.
#pragma once

#include "common.cuh"

namespace ge {

constexpr int kF8Block = 128;  // columns that share a scale: one k-block, one 128-byte swizzle row

struct Fp8Params {
  CUtensorMap tmA, tmB;    // (K, M), (K, N): boxes of 128 bytes by 128 rows (A) and BN / CG (B)
  uint32_t *status;
  uint64_t timeout_ns;
  const float *sa, *sb;    // [k-block][row], [k-block][column or column block]
  int64_t lds_a, lds_b;
  const void *c;           // added, or nullptr
  void *d;
  float *part;             // slices: [slice][M][ld_part] sums instead of D
  int64_t ldd, ld_part;
  int32_t M, N;
  int32_t num_kb, num_m_blk, num_n_blk, raster_group;
  int32_t slices, kb_split;  // a tile's k-blocks are shared by `slices` units, kb_split each
  int32_t stages;
  int32_t a_e5m2, b_e5m2, dt, vec;  // vec: rows of C and D are whole 32-byte units
  int32_t a_rows;          // rows of an A tile that are loaded (one CTA)
  uint32_t debug_flags;
  uint32_t off_B, off_bar;
};

constexpr int kF8Threads = 32 * (2 + 8);  // producer, MMA, 8 epilogue warps
constexpr uint32_t kF8BarBytes = 256;
// B's row scales of a k-block, a copy for each epilogue warp of its half of the columns, two deep
__host__ __device__ constexpr uint32_t fp8_scale_bytes(int bn) { return 8u * 2u * static_cast<uint32_t>(bn / 2) * 4u; }

// square: B's scales are one for each 128 columns
const void *fp8_kernel_cg1(bool square);  // 128 x 128 tiles, one CTA
const void *fp8_kernel_cg2(bool square);  // 256 x 256 tiles, a CTA pair

}  // namespace ge
