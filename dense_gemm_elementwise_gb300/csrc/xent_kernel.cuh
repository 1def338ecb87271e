// xent_kernel.cuh -- the products of the vocabulary loss on sm_103a.
//
// One persistent, warp-specialised kernel in five modes (XentMode):
//   X_STATS   H @ W^T, K-major operands: logits that never leave the SM.  An
//             epilogue thread owns one row of the tile and half of its
//             columns, which it holds in registers: it takes their maximum, then
//             the sum of 2^(x - maximum), and leaves the pair for the kernel
//             that joins the tiles.
//   X_KEEP    the same, and each logit's distance below that maximum in 16 bits,
//             from which dl is made without the product of X_DLOGIT.
//   X_DLOGIT  the same product: 2^(x - lse) * coef, less the target's 1, rounded
//             to 16 bits into the piece buffer.
//   X_OUT     dl^T @ H: dl read M-major, H N-major, the accumulator times one
//             scale into dW.
//   X_PART    dl @ W: dl K-major, W N-major, fp32 sums into slices, one
//             per range of K (few rows make few tiles: K is split over the
//             SMs), added by the TMA engine to earlier pieces' sums.  One
//             tile of a launch owns each element of its slice, so the order
//             of the additions is that of the launches.
// Warps: 0 loads operands (TMA, an S-stage ring), 1 allocates TMEM and issues
// tcgen05.mma into one of two accumulators, 2..9 are two epilogue groups of
// four warps that take the tile's column steps in turn, a thread to a row.  The number of rows that
// take part is read from device memory, so a batch with ignored targets costs
// what its other rows cost.  Mainloop and roles follow gemm_kernel.cuh.
//
// The products are bound by the tensor pipe when the batch is long and by
// reading W when it is short.
//
// Every wait is bounded, as in gemm_kernel.cuh: an epilogue group agrees on the
// outcome of its wait before its next barrier, so none of its warps is left alone.
#pragma once

#include "gemm_kernel.cuh"
#include "xent.cuh"
#include "xent_math.cuh"

namespace ge {

__device__ __forceinline__ void group_barrier(int id) {
  __syncwarp();
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
  __syncwarp();
}

// whether every thread of the group says yes
__device__ __forceinline__ bool group_agrees(int id, bool yes) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(yes ? 1u : 0u)
      : "memory");
  __syncwarp();
  return r != 0;
}

__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap *m, uint32_t src, int32_t x, int32_t y,
                                                  int32_t z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::
                   "l"(reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// 16 values of 16 bits to global memory: 32 bytes at once where they are aligned so
__device__ __forceinline__ void st_global32(uint16_t *p, const uint32_t *w, bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// barrier block
constexpr uint32_t kXFull = 0, kXEmpty = 64, kXTmemFull = 128, kXTmemEmpty = 144, kXDrain = 160,
                   kXTmemSlot = 168, kXAbort = 172;

struct XentTile {
  int z, mb, nb, kb0, kb1;
  int n0, width;  // first column and columns
};

template <int CG, int BN, int MODE>
__global__ void __launch_bounds__(kXentThreads, 1) xent_kernel(const __grid_constant__ XentParams p) {
  using T = TileCfg<CG, BN>;
  constexpr bool kAmn = MODE == X_OUT;                      // A is M-major
  constexpr bool kStats = MODE == X_STATS || MODE == X_KEEP;
  constexpr bool kBk = kStats || MODE == X_DLOGIT;           // B is K-major
  constexpr int kEpi0 = 2;                                   // first epilogue warp
  // k-blocks that the tensor unit sums before the epilogue adds them up in
  // registers.  Its sums are cut off, not rounded: left to itself over all of K it gives an
  // lse that is low by 2.0e-6 of its value at D = 4096 and 4.0e-6 at 8192 (bf16: 4.8e-10 for every column;
  // fp16, whose products have more bits to lose: 5.9e-10), in runs of K = 1024 and of 832 by 5.0e-7
  // whatever D is.  (Runs of 1536 lose 7.4e-7 and 8.8e-7, and save 2 % of a step at D = 1280; runs of 256 lose
  // 1.2e-7, but their 2000 clocks are less than their sums take to be read: 4096 x 65536 x 2048 in
  // 24 % more time.)
  const int most_run = p.bf16 ? 16 : 13;
  constexpr int kTogether = 2;  // k-blocks loaded together in bands
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG > 1 ? cluster_ctarank() : 0u;
  const int unit = blockIdx.x / CG, n_units = gridDim.x / CG;
  const uint32_t bar = sb + p.off_bar;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + p.off_bar + kXTmemSlot);
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + p.off_bar + kXAbort);

  if (warp == 0) {
    if (lane < p.stages) {
      mbar_init(bar + kXFull + 8 * lane, 1);
      mbar_init(bar + kXEmpty + 8 * lane, 1);
    }
    if (lane < 2) {
      mbar_init(bar + kXTmemFull + 8 * lane, 1);
      mbar_init(bar + kXTmemEmpty + 8 * lane, 8 * CG);
    }
    if (lane == 0) {
      mbar_init(bar + kXDrain, 1);
      *abort_flag = 0u;
      prefetch_tensormap(&p.tmA);
      prefetch_tensormap(&p.tmB);
    }
    fence_mbarrier_init();
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc<CG>(smem_u32(tmem_slot), T::kTmemCols);
    tmem_relinquish<CG>();
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (CG > 1) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
  griddep_wait();

  const Waiter wt{abort_flag, p.status, p.timeout_ns};
  const int rows = p.rows ? __ldcg(p.rows) : p.M;
  if (kStats && blockIdx.x == 0 && threadIdx.x == 0) p.sc->ticket = 0;  // of the kernel that follows
  const int M = MODE == X_OUT ? p.M : min(rows, p.M);
  const int num_m_blk = (M + T::kMmaM - 1) / T::kMmaM;
  // with no rows dW is 0: one k-block is run and its product dropped
  const int num_kb = MODE == X_OUT ? max(1, (min(rows, p.K) + BK - 1) / BK) : (p.K + BK - 1) / BK;
  const int per_slice = num_m_blk * p.num_n_blk;
  // dH's last tiles, too few for a wave of CTAs, are split along K; dW's along N
  const int kb_split = MODE == X_PART ? __ldcg(&p.sc->kb_split) : num_kb;
  const int num_full = MODE == X_PART ? min(per_slice, __ldcg(&p.sc->full))
                       : MODE == X_OUT && CG == 2 ? min(per_slice, p.num_full) : per_slice;
  const int rest = per_slice - num_full;
  const int num_tiles = num_full + rest * (MODE == X_PART ? (num_kb + kb_split - 1) / kb_split : 2);
  // (Runs of equal length: a short last one would be waited for.)
  const int runs = kStats ? (num_kb + most_run - 1) / most_run : 1;
  const int run = kStats ? (num_kb + runs - 1) / runs : num_kb;
  // In bands: unit u takes columns [u band, (u + 1) band) in tiles of up to BN.
  const bool bands = kStats && CG == 1 && p.band > 0;
  const int band_cols = bands ? max(0, min(p.band, p.N - unit * p.band)) : 0;
  const int my_tiles = bands ? (band_cols + BN - 1) / BN * num_m_blk
                             : unit < num_tiles ? (num_tiles - 1 - unit) / n_units + 1 : 0;
  auto tile = [&](int i) {
    XentTile t;
    if (bands) {
      t.z = t.mb = t.kb0 = 0;
      t.kb1 = num_kb;
      t.nb = unit * p.band_tiles + i;
      t.n0 = unit * p.band + i * BN;
      t.width = min(BN, p.band - i * BN);
      return t;
    }
    int at = unit + i * n_units, half = -1;
    const bool split = at >= num_full;
    t.z = 0;
    if (split) {
      const int j = at - num_full;
      if (MODE == X_PART) {
        t.z = j / rest;
        at = num_full + j - t.z * rest;
      } else {
        half = j & 1;
        at = num_full + (j >> 1);
      }
    }
    int batch;
    tile_coords(num_m_blk, p.num_n_blk, p.raster_group, at, batch, t.mb, t.nb);
    t.kb0 = MODE == X_PART && split ? t.z * kb_split : 0;
    t.kb1 = MODE == X_PART && split ? min(num_kb, t.kb0 + kb_split) : num_kb;
    t.n0 = t.nb * BN + (half > 0 ? BN / 2 : 0);
    t.width = half < 0 ? BN : BN / 2;
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      int stage = 0, fills = 0, skipped = -1;
      uint32_t phase = 0;
      bool ok = true, skip = (p.debug_flags & GE_DEBUG_SKIP_FIRST_LOAD) != 0u;
      auto next_stage = [&]() {
        ++fills;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      };
      // rows of H: packed, or H as it is
      const bool packed = rows < p.all_rows;
      const CUtensorMap *mA = kBk && !packed ? &p.tmH : &p.tmA, *mB = MODE == X_OUT && !packed ? &p.tmH : &p.tmB;
      for (int i = 0; ok && i < my_tiles; ++i) {
        const XentTile t = tile(i);
        const int m0 = t.mb * T::kMmaM + static_cast<int>(rank) * BM;
        const int n0 = t.n0 + static_cast<int>(rank) * (t.width / CG);
        const int nk = t.kb1 - t.kb0;
        if (bands) {
          // Two k-blocks together, so that memory is asked for 256 bytes of each row at
          // a time: 37 x 50001 x 2001 in 44.8 us against 47.2 one by one and 45.6 in threes
          // (half of the ring).  Whole tiles by boxes of 128 rows of W, others of 32.
          for (int kb = 0; ok && kb < nk; kb += kTogether) {
            const int some = min(kTogether, nk - kb);
            int at[kTogether], kq[kTogether];
#pragma unroll
            for (int q = 0; q < kTogether; ++q) {
              at[q] = kq[q] = -1;
              if (q >= some || !ok) continue;
              ok = wt.wait(bar + kXEmpty + 8 * stage, phase ^ 1u, SITE_PRODUCER_EMPTY);
              if (!ok) continue;
              if (skip) {
                skip = false;
                skipped = fills;
              } else {
                at[q] = stage;
                kq[q] = (i & 1) ? nk - 1 - kb - q : kb + q;
                const uint32_t full = bar + kXFull + 8 * stage;
                mbar_arrive_expect_tx(full, p.a_rows * 128 + t.width * 128);
                tma_load_3d(sb + stage * T::kABytes, mA, full, kq[q] * BK, m0, 0);
              }
              next_stage();
            }
            if (t.width == BN) {
#pragma unroll
              for (int q = 0; q < kTogether; ++q)
                if (at[q] >= 0)
                  tma_load_3d(sb + p.off_B + at[q] * T::kBBytes, mB, bar + kXFull + 8 * at[q], kq[q] * BK, n0, 0);
            } else {
              for (int j = 0; j < t.width; j += 32)
#pragma unroll
                for (int q = 0; q < kTogether; ++q)
                  if (at[q] >= 0)
                    tma_load_3d(sb + p.off_B + at[q] * T::kBBytes + j * 128, &p.tmB32, bar + kXFull + 8 * at[q],
                                kq[q] * BK, n0 + j, 0);
            }
          }
          continue;
        }
        for (int kb = 0; kb < nk; ++kb) {
          if (!wt.wait(bar + kXEmpty + 8 * stage, phase ^ 1u, SITE_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          if (skip) {
            skip = false;
            skipped = fills;
            next_stage();
            continue;
          }
          // odd tiles walk K backwards: a wave starts on what the last one left in L2
          const int kx = (t.kb0 + ((i & 1) ? nk - 1 - kb : kb)) * BK;
          const uint32_t full = bar + kXFull + 8 * stage;
          const uint32_t sa = sb + stage * T::kABytes, sbb = sb + p.off_B + stage * T::kBBytes;
          uint32_t fb = full;
          if constexpr (CG == 2) {
            fb = mapa_shared(full, 0);
            if (rank == 0) mbar_arrive_expect_tx(full, CG * T::kABytes + t.width * 128);
          } else {
            // few rows: only theirs are loaded; what the others' accumulators then hold is not read
            mbar_arrive_expect_tx(full, (kAmn ? T::kABytes : p.a_rows * 128) + T::kBBytes);
          }
          auto load = [&](uint32_t dst, const CUtensorMap *m, int x, int y) {
            if constexpr (CG == 2) tma_load_3d_pair(dst, m, fb, x, y, 0);
            else tma_load_3d(dst, m, fb, x, y, 0);
          };
          if constexpr (kAmn) {
            load(sa, mA, m0, kx);
            load(sa + 8192, mA, m0 + 64, kx);
          } else {
            load(sa, mA, kx, m0);
          }
          if constexpr (kBk) {
            load(sbb, mB, kx, p.b_row0 + n0);
          } else {
            // dH: the k rows of B are the piece's vocabulary rows
            const int ky = MODE == X_PART ? p.b_row0 + kx : kx;
#pragma unroll
            for (int j = 0; j < T::kBAtoms; ++j)
              if (64 * j < t.width / CG) load(sbb + j * 8192, mB, n0 + 64 * j, ky);
          }
          next_stage();
        }
      }
      // (at the start instead: no faster, 1 to 2 % slower on short batches)
      griddep_launch_dependents();
      if (ok) {
        for (int i = 0; i < p.stages; ++i) {
          if (!wt.wait(bar + kXEmpty + 8 * stage, phase ^ 1u, SITE_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && rank == 0) {
        for (int f = max(fills - p.stages, 0); f < fills; ++f)
          if (f != skipped)
            wt.drain(bar + kXFull + 8 * (f % p.stages), static_cast<uint32_t>(f / p.stages) & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    if (lane == 0 && rank == 0) {
      constexpr uint32_t kAk16 = (kAmn ? 2048u : 32u) >> 4, kBk16 = (kBk ? 32u : 2048u) >> 4;
      const uint64_t a_desc0 = smem_desc_sw128(sb, kAmn ? 8192u : 16u, 1024u);
      const uint64_t b_desc0 = smem_desc_sw128(sb + p.off_B, kBk ? 16u : 8192u, 1024u);
      int stage = 0, abuf = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        const XentTile t = tile(i);
        const uint32_t id = make_idesc_f16(p.bf16 != 0, T::kMmaM, t.width, kAmn, !kBk);
        for (int first = t.kb0; ok && first < t.kb1; first += run) {
          if (!wt.wait<CG == 2>(bar + kXTmemEmpty + 8 * abuf, aphase ^ 1u, SITE_MMA_TMEM_EMPTY)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(abuf * BN);
          const int end = min(t.kb1, first + run);
          for (int kb = first; kb < end; ++kb) {
            if (!wt.wait(bar + kXFull + 8 * stage, phase, SITE_MMA_FULL)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = a_desc0 + static_cast<uint32_t>(stage * (T::kABytes >> 4));
            const uint64_t bd = b_desc0 + static_cast<uint32_t>(stage * (T::kBBytes >> 4));
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
              umma_f16<CG>(d, ad + kAk16 * k, bd + kBk16 * k, id, (kb > first || k != 0) ? 1u : 0u);
            umma_commit<CG>(bar + kXEmpty + 8 * stage);
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          umma_commit<CG>(bar + kXTmemFull + 8 * abuf);
          abuf ^= 1;
          if (abuf == 0) aphase ^= 1u;
        }
      }
      if (ok) {
        for (int i = 0; i < 2; ++i) {
          if (!wt.wait<CG == 2>(bar + kXTmemEmpty + 8 * abuf, aphase ^ 1u, SITE_MMA_TMEM_EMPTY)) break;
          abuf ^= 1;
          if (abuf == 0) aphase ^= 1u;
        }
      } else {
        umma_commit<CG>(bar + kXDrain);
        wt.drain(bar + kXDrain, 0u);
      }
    }
  } else {
    // --------------------------------------------------------- epilogue --
    const int q = warp & 3;                   // TMEM lane quarter
    const int grp = (warp - kEpi0) >> 2;      // takes column steps grp, grp + 2, ...
    const int bid = 1 + grp;                  // the group's barrier
    const bool storer = ((warp - kEpi0) & 3) == 0 && lane == 0;
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const int row = q * 32 + lane;            // of the CTA's 128 accumulator rows
    const uint32_t sw = static_cast<uint32_t>(row & 7);
    const uint32_t boxes = sb + p.off_out + grp * kXentBoxes * kXentBox;
    int abuf = 0, step = 0;
    uint32_t aphase = 0;
    for (int i = 0; i < my_tiles; ++i) {
      const XentTile t = tile(i);
      const int m = t.mb * T::kMmaM + static_cast<int>(rank) * BM + row;
      const int n0 = t.n0;
      bool live = m < M;
      // what the row needs, on its way while the tile's product finishes
      int target = -1;
      float lse2 = 0.f, out_scale = 0.f;
      float2 coef = make_float2(0.f, 0.f);
      if ((kStats || MODE == X_DLOGIT) && live) {
        const int64_t at = p.target_i64 ? static_cast<const int64_t *>(p.target)[m] : static_cast<const int32_t *>(p.target)[m];
        // no column of this tile for a target that is elsewhere (or does not exist)
        if (MODE == X_DLOGIT && at < 0) live = false;
        const int64_t off = at - p.b_row0 - n0;
        target = off >= 0 && off < t.width ? static_cast<int>(off) : -1;
      }
      if (MODE == X_DLOGIT && live) {
        const float ds = p.sc->dl_scale;
        lse2 = p.lse2[m];
        coef = p.coef[m];
        coef.x *= ds;
        coef.y *= ds;
      }
      if (MODE == X_OUT) out_scale = rows > 0 ? *p.out_scale : 0.f;
      const int limit = p.N - n0;  // columns of the tile that exist
      // the accumulator is complete: no where the wait ran out
      auto ready = [&]() {
        const bool got = wt.wait(bar + kXTmemFull + 8 * abuf, aphase, SITE_EPI_TMEM_FULL);
        if (!group_agrees(bid, got)) return false;
        tc_fence_after();
        return true;
      };
      // it has been read: the next one
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t tb = bar + kXTmemEmpty + 8 * abuf;
          if constexpr (CG == 2) mbar_arrive_remote(mapa_shared(tb, 0));
          else mbar_arrive(tb);
        }
        abuf ^= 1;
        if (abuf == 0) aphase ^= 1u;
      };

      if constexpr (kStats) {
        // this group's columns, 64 of every 128, in registers
        constexpr int kParts = BN / 64;  // of 32 columns: grp * 64 + 128 (j / 2) + 32 (j % 2)
        float v[kParts][32];
        auto part = [&](int j) { return 128 * (j / 2) + 32 * (j % 2); };
        bool ok = ready();
        if (!ok) break;
        {  // the first run: all loads on their way at once
          const uint32_t acc = tq + static_cast<uint32_t>(abuf * BN + grp * 64);
#pragma unroll
          for (int j = 0; j < kParts; ++j) {
            tmem_ld16(acc + part(j), *reinterpret_cast<float(*)[16]>(v[j]));
            tmem_ld16(acc + part(j) + 16, *reinterpret_cast<float(*)[16]>(v[j] + 16));
          }
          tmem_wait_ld();
          release();
        }
        for (int first = t.kb0 + run; first < t.kb1; first += run) {
          if (!(ok = ready())) break;
          const uint32_t acc = tq + static_cast<uint32_t>(abuf * BN + grp * 64);
#pragma unroll
          for (int j = 0; j < 2 * kParts; ++j) {
            float x[16];
            tmem_ld16(acc + part(j / 2) + 16 * (j % 2), x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[j / 2][16 * (j % 2) + e] += x[e];
          }
          release();
        }
        if (!ok) break;
        const bool upside = p.c2 >= 0.f;  // the largest logit is the largest product, or the least
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
          const int c0 = grp * 64 + part(j);
          const int at = target - c0;
          if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e) x = at == e ? v[j][e] : x;
            if (at >= 0 && at < 32 && target < limit) p.at_target[m] = x * p.c;
          }
          const int end = min(limit, t.width) - c0;
          if (end < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= end) v[j][e] = upside ? -INFINITY : INFINITY;
          }
        }
        float top = upside ? -INFINITY : INFINITY;
        if (upside) {
#pragma unroll
          for (int j = 0; j < kParts; ++j)
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fmaxf(top, v[j][e]);
        } else {
#pragma unroll
          for (int j = 0; j < kParts; ++j)
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fminf(top, v[j][e]);
        }
        // rounded up: no distance below it is negative, whose code would wrap to the farthest (rounded to the
        // nearest, that took the maximum itself from a fifth of the rows with logits of 3000)
        top = __fmul_ru(top, p.c2);
        const float off = top == -INFINITY ? 0.f : top;
        const bool keep = MODE == X_KEEP && live;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[j][e] = fmaf(v[j][e], p.c2, -off);
          const int c0 = grp * 64 + part(j);
          if (keep && keeps(n0, c0, t.width, p.keep_cols)) {
            // the distances, rounded to integers in the low bits of floats of 2^23 and more
            constexpr float k0 = 8388608.f, kStepsPerOctave = 1 << kKeptBits;
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float a = fminf(fmaf(v[j][2 * e], -kStepsPerOctave, k0), k0 + 65535.f);
              const float b = fminf(fmaf(v[j][2 * e + 1], -kStepsPerOctave, k0), k0 + 65535.f);
              w[e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
            }
            uint16_t *o = p.out + int64_t(m) * p.ld_out + n0 + c0;
            st_global32(o, w, true);
            st_global32(o + 16, w + 8, true);
          }
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            s0 += ex2(v[j][e]);
            s1 += ex2(v[j][e + 1]);
            s2 += ex2(v[j][e + 2]);
            s3 += ex2(v[j][e + 3]);
          }
          sum += (s0 + s1) + (s2 + s3);
        }
        if (live) p.stats[(2 * int64_t(t.nb) + grp) * p.M + m] = make_float2(top, sum);
      } else if constexpr (MODE == X_PART) {
        if (!ready()) break;
        const uint32_t acc = tq + static_cast<uint32_t>(abuf * BN);
        // boxes of 128 rows of 32 columns, which the TMA engine stores or adds
        for (int c0 = grp * 32; c0 < BN; c0 += 64, ++step) {
          const uint32_t box = boxes + (step & 1) * kXentBox;
          if (storer) bulk_wait_group_read<kXentBoxes - 1>();
          group_barrier(bid);  // the box has been read by its last store
          float v[32];
          tmem_ld16(acc + c0, *reinterpret_cast<float(*)[16]>(v));
          tmem_ld16(acc + c0 + 16, *reinterpret_cast<float(*)[16]>(v + 16));
          tmem_wait_ld();
          if (c0 + 64 >= BN) release();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared16(box + row * 128 + ((static_cast<uint32_t>(j) ^ sw) << 4), __float_as_uint(v[4 * j]),
                        __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
          fence_proxy_async_smem();
          group_barrier(bid);
          if (storer) {
            const int y = t.mb * T::kMmaM + static_cast<int>(rank) * BM;
            if (n0 + c0 < p.N) {
              if (p.accumulate) tma_reduce_add_3d(&p.tmOut, box, n0 + c0, y, t.z);
              else tma_store_3d(&p.tmOut, box, n0 + c0, y, t.z);
            }
            bulk_commit_group();
          }
        }
      } else {
        // A thread writes its row's columns itself, 32 bytes at a time: whole sectors,
        // and nothing that the warps of a group have to wait for.  (Through boxes in shared
        // memory, with a fence and two barriers for every 64 columns, a tile's epilogue took
        // about 12000 clocks, longer than 17 k-blocks' products.)
        if (!ready()) break;
        const uint32_t acc = tq + static_cast<uint32_t>(abuf * BN);
        for (int c0 = grp * 32; c0 < t.width; c0 += 64) {
          float v[32];
          tmem_ld16(acc + c0, *reinterpret_cast<float(*)[16]>(v));
          tmem_ld16(acc + c0 + 16, *reinterpret_cast<float(*)[16]>(v + 16));
          tmem_wait_ld();
          if (c0 + 64 >= t.width) release();
          if constexpr (MODE == X_DLOGIT) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = ex2(fmaf(v[e], p.c2, -lse2)) * coef.x;
            const int at = target - c0;
            if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (at == e) v[e] -= coef.y;
            }
            // rows and columns that do not exist read as 0 in the products to come
            if (!live || c0 + 32 > limit) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!live || c0 + e >= limit) v[e] = 0.f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = rows > 0 ? v[e] * out_scale : 0.f;
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack16(p.bf16, v[2 * e], v[2 * e + 1]);
          // dl has zero rows up to the tile's last, as far as the buffer goes
          if (m >= (MODE == X_DLOGIT ? p.M : M)) continue;
          uint16_t *o = p.out + (MODE == X_OUT ? int64_t(p.b_row0) + m : int64_t(m)) * p.ld_out + n0 + c0;
          if (MODE == X_DLOGIT || c0 + 32 <= limit) {
            st_global32(o, w, MODE == X_DLOGIT || p.out32);
            st_global32(o + 16, w + 8, MODE == X_DLOGIT || p.out32);
          } else {
            // the last columns: 16 bytes at a time as far as they go (one by one, each row's
            // elements cost as much as the 32 bytes of the others)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (c0 + 8 * u + 8 <= limit) {
                *reinterpret_cast<uint4 *>(o + 8 * u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
              } else {
#pragma unroll
                for (int e = 8 * u; e < 8 * u + 8; ++e)
                  if (c0 + e < limit) o[e] = static_cast<uint16_t>(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
              }
            }
          }
        }
      }
    }
    // ranges of a band that have no columns
    if (bands && row < M)
      for (int i = my_tiles; i < p.band_tiles; ++i)
        p.stats[(2 * (int64_t(unit) * p.band_tiles + i) + grp) * p.M + row] = make_float2(-INFINITY, 0.f);
    if (MODE == X_PART && storer) bulk_wait_group<0>();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown --
  __syncwarp();
  tc_fence_before();
  if constexpr (CG > 1) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, T::kTmemCols);
  }
}

template <int CG, int BN>
const void *pick_xent(int mode) {
  switch (mode) {
    case X_STATS: return reinterpret_cast<const void *>(xent_kernel<CG, BN, X_STATS>);
    case X_DLOGIT: return reinterpret_cast<const void *>(xent_kernel<CG, BN, X_DLOGIT>);
    case X_OUT: return reinterpret_cast<const void *>(xent_kernel<CG, BN, X_OUT>);
    case X_PART: return reinterpret_cast<const void *>(xent_kernel<CG, BN, X_PART>);
    case X_KEEP: return reinterpret_cast<const void *>(xent_kernel<CG, BN, X_KEEP>);
    default: return nullptr;
  }
}

}  // namespace ge
