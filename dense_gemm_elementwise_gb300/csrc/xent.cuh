// xent.cuh -- parameters and handles of the vocabulary loss's products.
#pragma once

#include "common.cuh"
#include "xent_bands.h"

namespace ge {

// What one product's epilogue does with its accumulator.
enum XentMode {
  X_STATS = 0,   // logits: each row's maximum and sum of exponentials, the target's logit
  X_DLOGIT = 1,  // logits again: their gradient, rounded, into the piece buffer
  X_OUT = 2,     // a gradient: scaled, rounded, stored (dW)
  X_PART = 3,    // fp32 partial sums (dH), stored or added to what is there
  X_KEEP = 4,    // X_STATS, and the logits' distances below their range's maximum, 16 bits each
};

// Device scalars of a run, at the start of the workspace.
struct XentScalars {
  int32_t rows;       // rows that take part
  int32_t ticket;     // finish blocks done
  int32_t full;       // dH: tiles [0, full) sum a whole piece, ...
  int32_t kb_split;   // ... the others slices of this many k-blocks
  float out_scale;    // multiplies dl @ W and dl^T @ H
  float dl_scale;     // power of two in dl
};

// A kept logit is its distance below its range's maximum in log2 units, in
// fixed point with 11 bits after the point: p comes out off by at most 2^-12 ln 2 =
// 1.7e-4, a twentieth of bf16's rounding (2^-8), and what is below 2^-32 of the maximum of
// its own 64 to 128 columns counts as 0.  fp16 rounds too finely for that
// (2^-11), so its logits are not kept but computed twice.
constexpr int kKeptBits = 11;

constexpr int kXentBoxes = 2;            // X_PART: output boxes per epilogue group
constexpr uint32_t kXentBox = 128 * 128; // one box: 128 rows of 128 bytes

struct XentParams {
  CUtensorMap tmA, tmB, tmOut;
  CUtensorMap tmB32;       // bands: B in boxes of 32 rows
  CUtensorMap tmH;         // H itself, read in the packed rows' place when every row takes part
  uint32_t *status;
  uint64_t timeout_ns;
  XentScalars *sc;
  const int32_t *rows;     // rows that take part (device); nullptr: all M
  int32_t all_rows;        // T
  int32_t M, N, K;         // sizes at most; the rows replace M (K for X_OUT)
  int32_t num_n_blk, raster_group;
  int32_t num_full;        // X_OUT: tiles [0, num_full) are whole, each later pair the column halves of one
  int32_t stages;
  uint32_t debug_flags;
  int32_t a_rows;          // rows of an A tile that are loaded (K-major A, one CTA)
  // X_STATS, X_KEEP of a single tile of rows: columns of a CTA's band (0: tiles dealt out) and its tiles
  int32_t band, band_tiles;
  int32_t bf16;
  int32_t b_row0;          // first vocabulary row of this piece
  int32_t accumulate;      // X_PART: add to the slices
  uint32_t off_B, off_out, off_bar;
  float c;                 // logit_scale
  float c2;                // logit_scale * log2(e)
  const void *target;      // the rows' targets (X_DLOGIT: below 0 for a row that takes no part), ...
  int32_t target_i64;      // ... 8 bytes each, as the caller has them (else 4)
  int32_t keep_cols;       // X_KEEP: columns that are kept
  float2 *stats;           // [2 * blocks of BN columns][M]: maximum (log2 units), sum
  float *at_target;        // ... the target's logit
  const float *lse2;       // ... log2-sum-exp2 of its logits
  const float2 *coef;      // ... factors of p and of the target's 1
  const float *out_scale;  // one float
  uint16_t *out;           // X_KEEP, X_DLOGIT: the piece buffer; X_OUT: dW
  int64_t ld_out;
  int32_t out32;           // X_OUT: its rows are whole 32-byte units
};

const void *xent_kernel_cg1(int mode);  // 128 x 128 tiles, one CTA
const void *xent_kernel_cg2(int mode);  // 256 x 256 tiles, a CTA pair
constexpr int kXentThreads = 32 * (2 + 8);  // producer, MMA, 8 epilogue warps

}  // namespace ge
