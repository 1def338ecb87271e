// norm.h -- parameters and handles of the norms around a block.
#pragma once

#include <stdint.h>

namespace ge {

constexpr int kChunk = 8;        // columns a thread holds per chunk
constexpr int kVecThreads = 512;   // threads of a CTA, at most
constexpr int kMaxThreads = 1024;  // ... with other rows than of whole 16-byte units
// The forward pass is held to the registers of a CTA of 768 (85), so that three CTAs of 256 share
// an SM: 8192 x 4096 bf16 in 45.0 us against 47.9 with two.  The gradients keep 128
// (139 us against 307 for 16384 x 4096, whose sums then spill).
constexpr int kRunBound = 768;
constexpr int kMaxAhead = 3;     // rows in the ring of a thread
constexpr int kSumBytes = 2 * (kMaxThreads / 32) * 16;  // shared memory of the rows' sums

struct NormParams {
  const void *x, *b, *gate, *w_post, *w_pre;
  void *y, *h;
  // gradients
  const void *dy, *dh, *yin;
  void *dx, *db, *dgate;
  float *part_pre, *part_post;  // [units][ld_part]
  int64_t ld_part;
  int64_t ldx, ldb, ldy, ldh;
  int64_t rows_per_gate;
  int32_t T, D, wt;
  int32_t pre, post;
  float eps_pre, eps_post, alpha, inv_d;
  int32_t row_threads;   // threads that share a row: a power of two up to 32, or whole warps
  int32_t ahead;         // rows of the ring
  int32_t w_vec;         // gate's rows and the vectors are whole 16-byte units
  // units of the gradient pass; rows_per_unit is also the forward pass's run of a CTA, 0: dealt out
  int32_t units, rows_per_unit, rows_per_lane;
  int32_t units_per_group;  // 0: a lane holds whole groups
};

// Kernels, by how rows are moved; nv chunks per thread (1 or 2; whole units also 4), `threads` of a CTA.
enum NormRows {
  ROWS_16 = 0,     // whole 16-byte units (nv 1, 2, 4)
  ROWS_SMALL = 1,  // even pitches, or odd ones of fp32 (`even` says which): 4 or 8 bytes at a time
  ROWS_ODD = 2,    // odd pitches of 16-bit elements, one by one
};
const void *norm_kernel_run(int dt, int nv);
const void *norm_kernel_grad(int dt, int nv);
const void *norm_kernel_grad_whole(int dt, int nv);  // units hold whole gate groups
const void *norm_kernel_run_small(int dt, int nv, int threads, bool even);
const void *norm_kernel_grad_small(int dt, int nv, int threads, bool even);
const void *norm_kernel_grad_whole_small(int dt, int nv, int threads, bool even);
const void *norm_kernel_run_odd(int dt, int nv, int threads);
const void *norm_kernel_grad_odd(int dt, int nv, int threads);
const void *norm_kernel_grad_whole_odd(int dt, int nv, int threads);

}  // namespace ge
