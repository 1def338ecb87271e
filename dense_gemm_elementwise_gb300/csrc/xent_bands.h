// xent_bands.h -- where the logits that X_KEEP leaves lie: bands, pieces, and what of a tile is kept.
// Plain C++, so that the arithmetic is tested on the CPU as it is compiled for the GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GE_HOST_DEVICE inline
#endif

namespace ge {

// Columns of a CTA's band, with `units` CTAs: a multiple of 32 that need not divide anything else.
inline int64_t band_of(int64_t V, int64_t units) {
  const int64_t steps = (V + 31) / 32;
  return 32 * ((steps + units - 1) / units);
}

// Columns of a piece of the vocabulary, which are also the row pitch of its buffer: pieces as wide as
// the buffer allows, equal, whole tiles (multiples of 256).
inline int64_t piece_of(int64_t T, int64_t V, int64_t buffer_bytes) {
  const int64_t fit = buffer_bytes / (2 * T) / 256 * 256, widest = fit > 256 ? fit : 256;
  const int64_t pieces = (V + widest - 1) / widest;
  return ((V + pieces - 1) / pieces + 255) / 256 * 256;
}

// Whether columns [c0, c0 + 32) of a tile of `width` columns that starts at column n0 are kept.  A band's tile
// can end past keep_cols, where the next row of the buffer begins; keep_cols and tiles are
// multiples of 32, so whole steps decide it.
GE_HOST_DEVICE bool keeps(int n0, int c0, int width, int keep_cols) {
  return c0 < width && n0 + c0 < keep_cols;
}

// Column ranges that leave a maximum and a sum: two to a tile of bn columns, its odd and even runs of 64.
inline int64_t slots_of(int64_t V, int64_t band, int64_t bn) {
  return band ? 2 * ((V + band - 1) / band) * ((band + bn - 1) / bn) : 2 * ((V + bn - 1) / bn);
}

// The range of column c, of N that exist.  Past them there is none, and the first is named:
// what is read of it is dropped.
GE_HOST_DEVICE int slot_of(int c, int N, int band, int band_tiles, int bn) {
  if (c >= N) return 0;
  const int of_band = band ? c % band : c;
  return 2 * ((band ? c / band * band_tiles : 0) + of_band / bn) + ((of_band / 64) & 1);
}

}  // namespace ge
