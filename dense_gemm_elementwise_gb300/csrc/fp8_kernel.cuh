// fp8_kernel.cuh -- the product of 8-bit floats with a scale for each block of 128, on sm_103a.
//
//   D = C + sum_j scale_a[j] scale_b[j] (A_j @ B_j^T)
//
// Persistent and warp-specialised: warp 0 loads operands (TMA, a ring of k-blocks of 128 bytes), warps 1 and
// 2 issue tcgen05.mma.kind::f8f6f4 (1 also allocates TMEM), warp 3 brings the scales, warps 4..11 hold the
// tile's sums.  The scales differ from k-block to k-block, so each k-block is a product of its own: it
// lands in one of two TMEM accumulators, and the epilogue warps add it, scaled, to fp32
// registers (a thread has one row and half of the tile's columns) while the tensor unit fills
// the other.  fp32 additions in registers are rounded, which the tensor unit's are not.
//
// That is a hand-over between the tensor unit and the epilogue for every 512 clocks of tensor work, whose
// latencies bound the kernel (8192^3: 441 us in a row, 2.49 PFLOP/s, under the power cap; in bursts 413, and 375 without hand-overs, one sum
// over all of K.  Times below are of bursts):
//   * Accumulators are handed back by arrivals without release and waited for without acquire; nothing
//     but tensor memory is passed on, which the tcgen05 fences order.  (975 -> 519 us: release and acquire at
//     cluster scope take about 1000 clocks each.)
//   * One commit for each k-block: a stage's "done" barrier tells the producer that the stage is
//     free and the epilogue that the accumulator is complete.  (It cannot be a phase ahead of an epilogue warp:
//     that takes the stage's next k-block, for which the warps have to hand back this accumulator.)
//   * Two threads issue, one for each accumulator: a k-block costs such a thread about 1000 clocks, most of
//     them the latencies of its looks at barriers and of its issues.  (Four accumulators of half the columns
//     took 490 us and more: A is then read twice from shared memory.)
//   * Scales come through shared memory, some k-blocks at a time: loaded by the epilogue itself, a
//     k-block ahead, they came too late (with constants in their place it took 30 us less).
//   * 32 columns (16) are on their way to an epilogue thread while it adds as many others, which its registers
//     have room for because the other warps give theirs away.  (Sixteen epilogue warps took 530 us.)
//   * The loop over a k-block has one way through it.  A second one, for scales whose product no normal fp32 number holds,
//     made the compiler spill in the first: 8192^3 in a row 437 -> 447 us where it was chosen for eight k-blocks at a time, 480 to
//     526 where for each.  So the range of the scales is the interface's.
//
// Few tiles (128 x 128, single CTAs) share their sums over K with the other CTAs of a cluster, which leave them in
// shared memory, where each CTA then adds its part of the tile in the order of the slices: one launch, no
// workspace (37 x 5001 x 2000 in 7.9 us; with slices in memory and a second launch 9.2).
//
// Every wait is bounded, as in gemm_kernel.cuh.  No epilogue warp waits for another.
#pragma once

#include "fp8.cuh"
#include "gemm_kernel.cuh"
#include "xent_math.cuh"

namespace ge {

// barrier block
constexpr uint32_t kFFull = 0, kFDone = 64, kFTmemEmpty = 128, kFDrain = 144, kFScaleFull = 160, kFScaleEmpty = 176,
                   kFTmemSlot = 192, kFAbort = 196;

// A wait that is short as a rule: the clock is looked at when it is not.
__device__ __forceinline__ bool wait_soon(const Waiter &wt, uint32_t bar, uint32_t parity, uint32_t site) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return wt.wait(bar, parity, site);
}

// the same for an accumulator that both CTAs of a pair hand back (see above)
__device__ __forceinline__ bool wait_soon_relaxed(const Waiter &wt, uint32_t bar, uint32_t parity, uint32_t site) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait_relaxed(bar, parity)) return true;
  return wt.wait<true>(bar, parity, site);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 8 words of a row, 32 bytes or twice 16 at a time
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = *static_cast<const uint4 *>(p), b = *(static_cast<const uint4 *>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

__device__ __forceinline__ void store_words(void *p, const uint32_t *w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *(static_cast<uint4 *>(p) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// C's 64 columns from `at` on added to as many sums: asked for together, since D may be C and no load passes a store
__device__ __forceinline__ void add64(const Fp8Params &p, int64_t at, float2 *sums) {
  if (p.dt == GE_F32) {
    uint32_t w[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load_words(static_cast<const float *>(p.c) + at + 8 * i, w[i], p.vec == 2);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sums[4 * i + e].x += __uint_as_float(w[i][2 * e]);
        sums[4 * i + e].y += __uint_as_float(w[i][2 * e + 1]);
      }
  } else {
    const bool bf16 = p.dt == GE_BF16;
    uint32_t w[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) load_words(static_cast<const uint16_t *>(p.c) + at + 16 * i, w[i], p.vec == 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 c = bf16 ? make_float2(__uint_as_float(w[i][e] << 16), __uint_as_float(w[i][e] & 0xffff0000u))
                              : __half22float2(*reinterpret_cast<const __half2 *>(&w[i][e]));
        sums[8 * i + e].x += c.x;
        sums[8 * i + e].y += c.y;
      }
  }
}

// 16 sums of a row, C added where `add`, into D
__device__ __forceinline__ void finish16(const Fp8Params &p, int m, int n, float (&v)[16], bool add) {
  const int left = p.N - n;
  const int64_t at = int64_t(m) * p.ldd + n;
  if (left >= 16) {  // (rows are whole 16 bytes)
    if (p.dt == GE_F32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[8];
        if (add) {
          load_words(static_cast<const float *>(p.c) + at + 8 * h, w, p.vec == 2);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[8 * h + e] += __uint_as_float(w[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[8 * h + e]);
        store_words(static_cast<float *>(p.d) + at + 8 * h, w, p.vec == 2);
      }
    } else {
      const bool bf16 = p.dt == GE_BF16;
      uint32_t w[8];
      if (add) {
        load_words(static_cast<const uint16_t *>(p.c) + at, w, p.vec == 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 c = bf16 ? make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u))
                                : __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
          v[2 * e] += c.x;
          v[2 * e + 1] += c.y;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = pack16(bf16, v[2 * e], v[2 * e + 1]);
      store_words(static_cast<uint16_t *>(p.d) + at, w, p.vec == 2);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < left) store_one(p.d, at + e, p.dt, v[e] + (add ? load_one(p.c, at + e, p.dt) : 0.f));
}

// How D is written: rows of whole 16 bytes without C, the same with C (a kernel of its own: the loads' registers took 2 % of the
// other's time), or rows that start anywhere
enum Fp8Out { kF8Plain, kF8Add, kF8Turn };

template <int CG, int BN, bool SQUARE, Fp8Out OUT>
__global__ void __launch_bounds__(kF8Threads, 1) fp8_kernel(const __grid_constant__ Fp8Params p) {
  using T = TileCfg<CG, BN>;
  constexpr int kEpi0 = kF8Epi0;
  constexpr int kCols = BN / 2;  // columns of an epilogue thread
  constexpr int kBatch = fp8_batch(SQUARE), kSb = SQUARE ? 2 : BN, kBatchFloats = kBatch * (128 + kSb);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG > 1 ? cluster_ctarank() : 0u;
  const int unit = blockIdx.x / CG, n_units = gridDim.x / CG;
  const uint32_t bar = sb + p.off_bar;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + p.off_bar + kFTmemSlot);
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + p.off_bar + kFAbort);

  if (warp == 0) {
    if (lane < p.stages) {
      mbar_init(bar + kFFull + 8 * lane, 1);
      mbar_init(bar + kFDone + 8 * lane, 1);
    }
    if (lane < 2) mbar_init(bar + kFTmemEmpty + 8 * lane, 8 * CG);
    if (lane < 2) {
      mbar_init(bar + kFDrain + 8 * lane, 1);
      mbar_init(bar + kFScaleFull + 8 * lane, 1);
      mbar_init(bar + kFScaleEmpty + 8 * lane, 8);
    }
    if (lane == 0) {
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
  const int num_units = p.num_m_blk * p.num_n_blk * p.slices;
  struct Tile { int z, m0, n0, kb0, kb1; };
  auto tile = [&](int at) {
    Tile t;
    const int whole = at / p.slices;
    t.z = at - whole * p.slices;
    int l, mb, nb;
    tile_coords(p.num_m_blk, p.num_n_blk, p.raster_group, whole, l, mb, nb);
    t.m0 = mb * T::kMmaM + static_cast<int>(rank) * BM;
    t.n0 = nb * BN;
    t.kb0 = t.z * p.kb_split;
    t.kb1 = min(p.num_kb, t.kb0 + p.kb_split);
    return t;
  };

  // (the registers that each side may use differ from here on: nothing runs on both before the end)
  if (warp < kEpi0) {
  set_registers<false, kF8RegsLess>();
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
      for (int at = unit; ok && at < num_units; at += n_units) {
        const Tile t = tile(at);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!wait_soon(wt, bar + kFDone + 8 * stage, phase ^ 1u, SITE_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          if (skip) {
            skip = false;
            skipped = fills;
            next_stage();
            continue;
          }
          const uint32_t full = bar + kFFull + 8 * stage;
          const uint32_t sa = sb + stage * T::kABytes, sbb = sb + p.off_B + stage * T::kBBytes;
          if constexpr (CG == 2) {
            const uint32_t fb = mapa_shared(full, 0);
            const int n0 = t.n0 + static_cast<int>(rank) * (BN / 2);
            if (rank == 0) mbar_arrive_expect_tx(full, CG * (T::kABytes + T::kBBytes));
            tma_load_3d_pair(sa, &p.tmA, fb, kb * kF8Block, t.m0, 0);
            tma_load_3d_pair(sbb, &p.tmB, fb, kb * kF8Block, n0, 0);
          } else {
            // few rows: only theirs are loaded; what the others' accumulators then hold is not read
            mbar_arrive_expect_tx(full, p.a_rows * 128 + T::kBBytes);
            tma_load_3d(sa, &p.tmA, full, kb * kF8Block, t.m0, 0);
            tma_load_3d(sbb, &p.tmB, full, kb * kF8Block, t.n0, 0);
          }
          next_stage();
        }
      }
      griddep_launch_dependents();
      if (ok) {
        for (int i = 0; i < p.stages; ++i) {
          if (!wait_soon(wt, bar + kFDone + 8 * stage, phase ^ 1u, SITE_PRODUCER_EMPTY)) {
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
          if (f != skipped) wt.drain(bar + kFFull + 8 * (f % p.stages), static_cast<uint32_t>(f / p.stages) & 1u);
      }
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------- MMA issuers --
    if (lane == 0 && rank == 0) {
      const uint64_t a_desc0 = smem_desc_sw128(sb, 16u, 1024u), b_desc0 = smem_desc_sw128(sb + p.off_B, 16u, 1024u);
      const uint32_t id = make_idesc_f8(p.a_e5m2 != 0, p.b_e5m2 != 0, T::kMmaM, BN);
      // this thread's accumulator takes every other k-block of the CTA's
      const int mine = warp - 1;
      const uint32_t d = tmem_base + static_cast<uint32_t>(mine * BN), empty = bar + kFTmemEmpty + 8 * mine;
      int stage = 0, count = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true;
      for (int at = unit; ok && at < num_units; at += n_units) {
        const Tile t = tile(at);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++count) {
          if ((count & 1) == mine) {
            if (!wait_soon(wt, bar + kFFull + 8 * stage, phase, SITE_MMA_FULL) ||
                !wait_soon_relaxed(wt, empty, aphase ^ 1u, SITE_MMA_TMEM_EMPTY)) {
              ok = false;
              break;
            }
            aphase ^= 1u;
            tc_fence_after();
            const uint64_t ad = a_desc0 + static_cast<uint32_t>(stage * (T::kABytes >> 4));
            const uint64_t bd = b_desc0 + static_cast<uint32_t>(stage * (T::kBBytes >> 4));
#pragma unroll
            for (int k = 0; k < kF8Block / 32; ++k) umma_f8<CG>(d, ad + 2 * k, bd + 2 * k, id, k != 0 ? 1u : 0u);
            umma_commit<CG>(bar + kFDone + 8 * stage);
          }
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (ok) {
        wt.wait<CG == 2>(empty, aphase ^ 1u, SITE_MMA_TMEM_EMPTY);
      } else {
        umma_commit<CG>(bar + kFDrain + 8 * mine);
        wt.drain(bar + kFDrain + 8 * mine, 0u);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ scales --
    float *buf = reinterpret_cast<float *>(smem + p.off_bar + kF8BarBytes);
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int at = unit; ok && at < num_units; at += n_units) {
      const Tile t = tile(at);
      const int es = p.dt == GE_F32 ? 4 : 2, lines = BN * es / 128;  // C's lines of a row
      int asked = OUT == kF8Add ? lane : BM * lines;
      for (int kb0 = t.kb0; kb0 < t.kb1; kb0 += kBatch) {
        // all of a batch's loads are under way before one is waited for
        float a[kBatch][4], b[SQUARE ? 1 : kBatch][SQUARE ? 1 : kSb / 32];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const bool on = kb0 + k < t.kb1;
          const float *sa = p.sa + int64_t(kb0 + k) * p.lds_a;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int m = t.m0 + 32 * i + lane;
            a[k][i] = on && m < p.M ? __ldg(sa + m) : 0.f;
          }
          if constexpr (!SQUARE) {
            const float *sbk = p.sb + int64_t(kb0 + k) * p.lds_b;
#pragma unroll
            for (int i = 0; i < kSb / 32; ++i) {
              const int n = t.n0 + 32 * i + lane;
              b[k][i] = on && n < p.N ? __ldg(sbk + n) : 0.f;
            }
          }
        }
        if constexpr (SQUARE) {
          const int n = t.n0 + (lane & 1) * kCols, k = kb0 + (lane >> 1);
          b[0][0] = lane < 2 * kBatch && n < p.N && k < t.kb1 ? __ldg(p.sb + int64_t(k) * p.lds_b + n / kF8Block) : 0.f;
        }
        ok = __all_sync(0xffffffffu, wait_soon(wt, bar + kFScaleEmpty + 8 * slot, phase ^ 1u, SITE_EPI_AUX_FULL));
        if (!ok) break;
        float *to = buf + slot * kBatchFloats;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) to[k * 128 + 32 * i + lane] = a[k][i];
          if constexpr (!SQUARE) {
#pragma unroll
            for (int i = 0; i < kSb / 32; ++i) to[kBatch * 128 + k * kSb + 32 * i + lane] = b[k][i];
          }
        }
        if (SQUARE && lane < 2 * kBatch) to[kBatch * 128 + lane] = b[0][0];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kFScaleFull + 8 * slot);
        slot ^= 1;
        if (slot == 0) phase ^= 1u;
        // some of C on its way to the L2 (all at once, the next scales came late)
#pragma unroll 1
        for (int i = 0; i < kBatch && asked < BM * lines; ++i, asked += 32) {
          const int m = t.m0 + asked / lines, n = t.n0 + asked % lines * (128 / es);
          if (m < p.M && n < p.N)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p.c) + (int64_t(m) * p.ldd + n) * es));
        }
      }
    }
  }
  } else {
    set_registers<true, kF8RegsMore>();
    // ---------------------------------------------------------- epilogue --
    const int q = warp & 3;             // TMEM lane quarter
    const int grp = (warp - kEpi0) >> 2;  // half of the columns
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(grp * kCols);
    const float *buf = reinterpret_cast<const float *>(smem + p.off_bar + kF8BarBytes);
    int abuf = 0, stage = 0, slot = 0;
    uint32_t phase = 0, sphase = 0;
    bool ok = true;
    for (int at = unit; ok && at < num_units; at += n_units) {
      const Tile t = tile(at);
      const int m = t.m0 + q * 32 + lane, n0 = t.n0 + grp * kCols;
      const bool live = m < p.M;
      float2 acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      int in_batch = 0;
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        if (in_batch == 0) {
          ok = __all_sync(0xffffffffu, wait_soon(wt, bar + kFScaleFull + 8 * slot, sphase, SITE_EPI_AUX_FULL));
          if (!ok) break;
        }
        const float *sa_now = buf + slot * kBatchFloats + in_batch * 128;
        const float *sb_now = buf + slot * kBatchFloats + kBatch * 128 + in_batch * kSb + (SQUARE ? grp : grp * kCols);
        float s = sa_now[q * 32 + lane];
        if constexpr (SQUARE) s *= *sb_now;
        const float2 s2 = make_float2(s, s);
        ok = __all_sync(0xffffffffu, wait_soon(wt, bar + kFDone + 8 * stage, phase, SITE_EPI_TMEM_FULL));
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tq + static_cast<uint32_t>(abuf * BN);
        auto back = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            const uint32_t tb = bar + kFTmemEmpty + 8 * abuf;
            if constexpr (CG == 2) mbar_arrive_remote_relaxed(mapa_shared(tb, 0));
            else mbar_arrive(tb);
          }
        };
        if constexpr (!SQUARE) {
          // 16 columns at a time leave registers for the next ones' scales, which then are there when their sums are (32 columns
          // without them: 4096 x 2048 x 6016 into fp32 69.2 us, here 67.9)
          float v[2][16];
          float4 b[2][4];
          tmem_ld16(src, v[0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) b[0][e] = *reinterpret_cast<const float4 *>(sb_now + 4 * e);
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            tmem_wait_ld();
            if (c + 1 < kCols / 16) {
              tmem_ld16(src + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) b[(c + 1) & 1][e] = *reinterpret_cast<const float4 *>(sb_now + 16 * (c + 1) + 4 * e);
            } else {
              back();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 w = b[c & 1][e];
              const float2 x = mul2(make_float2(v[c & 1][4 * e], v[c & 1][4 * e + 1]), make_float2(w.x, w.y));
              const float2 y = mul2(make_float2(v[c & 1][4 * e + 2], v[c & 1][4 * e + 3]), make_float2(w.z, w.w));
              acc[8 * c + 2 * e] = fma2(x, s2, acc[8 * c + 2 * e]);
              acc[8 * c + 2 * e + 1] = fma2(y, s2, acc[8 * c + 2 * e + 1]);
            }
          }
        } else {
          // 32 columns are on their way while the 32 before them are added
          float v[2][32];
          tmem_ld32(src, v[0]);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            tmem_wait_ld();
            if (c + 1 < kCols / 32) tmem_ld32(src + 32 * (c + 1), v[(c + 1) & 1]);
            else back();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              acc[16 * c + e] = fma2(make_float2(v[c & 1][2 * e], v[c & 1][2 * e + 1]), s2, acc[16 * c + e]);
          }
        }
        abuf ^= 1;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++in_batch == kBatch || kb + 1 == t.kb1) {
          in_batch = 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar + kFScaleEmpty + 8 * slot);
          slot ^= 1;
          if (slot == 0) sphase ^= 1u;
        }
      }
      if (!ok) break;
      if (OUT == kF8Turn && !(CG == 1 && p.slices > 1)) {
        // Rows that start anywhere: 32 columns of 32 rows through shared memory, so that a warp writes a row's
        // columns together (4096 x 10473 x 393 bf16: 353 us when each thread wrote its own row)
        float *turn = reinterpret_cast<float *>(smem + p.off_turn) + (warp - kEpi0) * 32 * kF8TurnPitch;
        const int m0 = t.m0 + q * 32, rows = min(32, p.M - m0);
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            turn[lane * kF8TurnPitch + 2 * e] = acc[16 * c + e].x;
            turn[lane * kF8TurnPitch + 2 * e + 1] = acc[16 * c + e].y;
          }
          __syncwarp();
          const int n = n0 + 32 * c + lane;
          if (n < p.N) {
#pragma unroll 8
            for (int r = 0; r < rows; ++r) {
              const int64_t at = int64_t(m0 + r) * p.ldd + n;
              store_one(p.d, at, p.dt, turn[r * kF8TurnPitch + lane] + (p.c ? load_one(p.c, at, p.dt) : 0.f));
            }
          }
        }
        continue;
      }
      if (!live) continue;
      if (CG == 1 && p.slices > 1) {  // the ring is free: all of this CTA's products are complete
        float *to = reinterpret_cast<float *>(smem) + (q * 32 + lane) * kF8PartPitch + grp * kCols;
#pragma unroll
        for (int e = 0; e < kCols / 2; e += 2)
          *reinterpret_cast<float4 *>(to + 2 * e) = make_float4(acc[e].x, acc[e].y, acc[e + 1].x, acc[e + 1].y);
        continue;
      }
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        const int n = n0 + 16 * c;
        if (n >= p.N) break;
        const bool whole = n0 + c / 4 * 64 + 64 <= p.N;
        if (OUT == kF8Add && c % 4 == 0 && whole) add64(p, int64_t(m) * p.ldd + n, acc + 8 * c);
        float v[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[2 * e] = acc[8 * c + e].x;
          v[2 * e + 1] = acc[8 * c + e].y;
        }
        finish16(p, m, n, v, OUT == kF8Add && !whole);
      }
    }
    __syncwarp();
  }

  if (CG == 1 && p.slices > 1) {
    // A cluster has one tile.  Its rows' groups of 4 columns are dealt out to the cluster's threads.  (After a
    // timeout what is added here is undefined, like the run's outputs.)
    __syncwarp();
    cluster_sync_all();
    const Tile t = tile(unit);
    const int rows = min(BM, p.M - t.m0), groups = rows * (BN / 4);
    for (int i = t.z * kF8Threads + static_cast<int>(threadIdx.x); i < groups; i += p.slices * kF8Threads) {
      const int r = i / (BN / 4), n = t.n0 + i % (BN / 4) * 4;
      const uint32_t at = sb + static_cast<uint32_t>(r * kF8PartPitch + i % (BN / 4) * 4) * 4u;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int z = 0; z < p.slices; ++z) {
        float4 x;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                     : "r"(mapa_shared(at, static_cast<uint32_t>(z)))
                     : "memory");
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      const float w[4] = {v.x, v.y, v.z, v.w};
      const int64_t out = int64_t(t.m0 + r) * p.ldd + n;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) store_one(p.d, out + e, p.dt, w[e] + (p.c ? load_one(p.c, out + e, p.dt) : 0.f));
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while its sums are read
  }

  // -------------------------------------------------------------- teardown --
  __syncwarp();
  tc_fence_before();
  if constexpr (CG > 1) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, T::kTmemCols);
  }
}

template <int CG, int BN, bool SQUARE>
const void *pick_fp8(bool add, bool turned) {
  return turned ? reinterpret_cast<const void *>(fp8_kernel<CG, BN, SQUARE, kF8Turn>)
         : add  ? reinterpret_cast<const void *>(fp8_kernel<CG, BN, SQUARE, kF8Add>)
                : reinterpret_cast<const void *>(fp8_kernel<CG, BN, SQUARE, kF8Plain>);
}

}  // namespace ge
