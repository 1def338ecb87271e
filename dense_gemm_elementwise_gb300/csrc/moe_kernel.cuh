// moe_kernel.cuh -- a mixture-of-experts layer for a few tokens (gemm_epi_moe_*): the experts' kernel; the
// router's, and where it has one the choice's, are in moe.cu.
//
//   router   l = x w_router^T, in pairs of fp32 (TwoSum): the choice of experts has to be that
//            of exact logits, or a token's output is another's
//   choice   of a token's experts, by a warp.  Where a CTA has a warp for each token, every CTA of the experts'
//            kernel chooses for itself (cheaper than a third launch or a grid-wide wait)
//   experts  CTAs take units of work by ticket:
//              1. 16 columns of h = act(gate) * up of one expert: 16 gate and 16 up rows against
//                 the tokens that chose it, up to 32 (more are another unit)
//              2. 32 columns of y's share of one expert: 32 rows of w_down against its h,
//                 times the routing weight; the last unit of those 32 columns adds the
//                 experts' shares in the order of the choice
//            A unit of the second kind waits for its expert's units of the first kind.
//            Tickets rise, so those are all held by CTAs that run and wait for nothing:
//            no CTA has to be resident for another to finish.
//
// Few tokens leave the tensor unit idle: the layer is bound by reading the chosen experts'
// weights once.  So a CTA's warps are there to keep that reading going:
//   producers take tickets and copy their rows, 1 KiB of 32 rows at a time, into a ring of
//             shared memory (cp.async, 16 bytes a lane), several units ahead of
//   consumers, a group or two of eight warps, which share a stage's columns and multiply them by mma.sync
//             (tcgen05 would want 128 rows of tokens): a lane reads 16 consecutive bytes of a row, and what it holds
//             is called columns 2q, 2q + 1, 2q + 8, 2q + 9 of a step; the tokens' side is read
//             the same way, so the sum runs over the same columns
//   watcher   waits for the h of units that are still on their way into the ring
//   finisher  tells the GPU that a unit is done.  Where it was the last one of its columns of y, their shares
//             are added by the producers, which have no more to copy by then, or by the finisher
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "moe.h"
#include "moe_choice.cuh"
#include "ptx.cuh"
#include "xent_math.cuh"

namespace ge {
namespace {

constexpr int kGroups = GE_MOE_GROUPS, kWarps = 8;  // consumers: groups of warps that share a unit, ...
constexpr int kProducers = 2;       // ... producers, each with half of the rows of every stage, ...
constexpr int kProducer = kGroups * kWarps, kWatcher = kProducer + kProducers, kFinisher = kWatcher + 1;  // watcher, finisher
constexpr int kThreads = 32 * (kFinisher + 1);
constexpr int kJobs = 4;            // columns of y whose shares are to be added, at most
constexpr int kBlock = 128;        // columns that share a scale
constexpr int kRows = 32, kRowTiles = kRows / 16;  // a unit's rows of weights
constexpr int kTile = 8;           // tokens of one mma
constexpr int kMostTokens = 32;    // of a unit
constexpr int kEntries = GE_MOE_MAX_EXPERTS + kPairs / kMostTokens;
constexpr int kRoundTiles = 1;     // of them whose sums are joined at a time
constexpr int kSegment = 1024;     // bytes of a row in a stage
constexpr int kPitch = kSegment + 64;  // lanes of two rows touch different banks
constexpr int kStages = 5;
constexpr int kQueue = 8;          // units under way in a CTA

// --------------------------------------------------------------- the lists --

struct Choice {
  uint16_t expert[kPairs];
  float weight[kPairs];
  uint16_t list[kPairs];             // pairs token * k + j, those of an expert together, ...
  uint8_t token[kPairs];             // ... and their tokens
  // experts that some token chose, once for every 32 pairs: how many of them, where in the list, and of how many entries
  uint16_t active[kEntries];
  uint8_t count[kEntries], parts[kEntries];
  uint16_t begin[kEntries];
  int32_t n_active;
  int32_t counter[GE_MOE_MAX_EXPERTS];
};

// The experts that some token chose, and each one's pairs.
__device__ void make_lists(const MoeParams &p, Choice &c) {
  const int pairs = p.T * p.k;
  for (int e = threadIdx.x; e < p.E; e += kThreads) c.counter[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kThreads) atomicAdd(&c.counter[c.expert[i]], 1);
  __syncthreads();
  if (threadIdx.x < 32) {
    int n = 0, at = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int k = e < p.E ? c.counter[e] : 0, parts = (k + kMostTokens - 1) / kMostTokens;
      int before = k, entries = parts;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, o), w = __shfl_up_sync(0xffffffffu, entries, o);
        if (static_cast<int>(threadIdx.x) >= o) before += v, entries += w;
      }
      for (int i = 0; i < parts; ++i) {
        const int a = n + entries - parts + i;
        c.active[a] = static_cast<uint16_t>(e);
        c.count[a] = static_cast<uint8_t>(min(kMostTokens, k - i * kMostTokens));
        c.parts[a] = static_cast<uint8_t>(parts);
        c.begin[a] = static_cast<uint16_t>(at + before - k + i * kMostTokens);
      }
      if (e < p.E) c.counter[e] = parts > 1 ? -1 : at + before - k;
      n += __shfl_sync(0xffffffffu, entries, 31);
      at += __shfl_sync(0xffffffffu, before, 31);
    }
    if (threadIdx.x == 0) c.n_active = n;
  }
  __syncthreads();
  // An expert's pairs in any order, another one in another CTA: each has a column of its own.  But those of several
  // entries have to be shared out alike by all CTAs: in order, by a warp.
  for (int i = threadIdx.x; i < pairs; i += kThreads)
    if (c.counter[c.expert[i]] >= 0) {
      const int at = atomicAdd(&c.counter[c.expert[i]], 1);
      c.list[at] = static_cast<uint16_t>(i);
      c.token[at] = static_cast<uint8_t>(i / p.k);
    }
  const int lane = threadIdx.x & 31;
  for (int a = threadIdx.x >> 5; a < c.n_active; a += kThreads / 32) {
    const int e = c.active[a];
    if (c.parts[a] == 1 || (a > 0 && c.active[a - 1] == e)) continue;
    int at = c.begin[a];
#pragma unroll 1
    for (int i0 = 0; i0 < pairs; i0 += 32) {
      const bool hit = i0 + lane < pairs && c.expert[i0 + lane] == e;
      const uint32_t hits = __ballot_sync(0xffffffffu, hit);
      const int place = at + __popc(hits & ((1u << lane) - 1u));
      if (hit) {
        c.list[place] = static_cast<uint16_t>(i0 + lane);
        c.token[place] = static_cast<uint8_t>((i0 + lane) / p.k);
      }
      at += __popc(hits);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- products --

template <int XT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (XT == GE_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two 8-bit floats, in the upper bytes of w's halves, as two values of type XT (exact, if they are finite).  To bf16 by
// shifting their bits into its exponent and mantissa, whose bias then is off by a power of two.
template <int XT, int WT>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  constexpr bool e4 = WT == GE_E4M3;
  if constexpr (XT == GE_BF16) {
    const uint32_t bits = ((w >> (e4 ? 4 : 3)) & (e4 ? 0x07f007f0u : 0x0fe00fe0u)) | (w & 0x80008000u);
    constexpr uint32_t by = e4 ? 0x7b807b80u : 0x77807780u;  // 2^120, 2^112
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&bits), *reinterpret_cast<const __nv_bfloat162 *>(&by));
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const uint16_t two = static_cast<uint16_t>(__byte_perm(w, 0, 0x4431));
    uint32_t h;
    if constexpr (e4) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(two));
    return h;
  }
}

// Whether one of four 8-bit floats is no finite number.  A row of weights that holds one gives NaN.  (The flags are looked
// at once for a unit: a branch for each 16 bytes took 905 us where this took 791, with 64 tokens and 128 experts of 4096 x 2048.)
template <int WT>
__device__ __forceinline__ uint32_t special(uint32_t w) {
  return WT == GE_E4M3 ? ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : ((w & 0x7c7c7c7cu) + 0x04040404u) & 0x80808080u;
}

// With one tile of tokens, the products with h and with what its rounding left have sums of their own: a
// chain of mma on one sum runs at their latency.
template <int NT, bool LO>
constexpr int kChains = NT == 1 && LO ? 2 : 1;

// Shapes of the products with a stage.
template <int WT, bool LO>
struct Shape {
  static constexpr bool k8 = WT == GE_E4M3 || WT == GE_E5M2;
  static constexpr int kPer = k8 ? 16 : 8;               // columns of a lane's 16 bytes
  static constexpr int kSteps = kSegment / 64 / kWarps;  // of 64 bytes of a row, for each warp: a scale's 128 columns
  static constexpr int kHalves = LO ? 2 : 1;
  static_assert(kSteps * 64 == 128, "a scale's columns; zeros are copied up to as many bytes");
  using Tokens = uint4[kSteps][kHalves][kPer / 8];       // the tokens' side of a step
};

// One token's side of this lane's columns of a stage, from `from` and, of what their rounding left, `rest` on; `bytes` of a
// row exist from the lane's first on (0 for a token that does not exist).  (h is written by other CTAs of this launch: no
// __ldg.)
template <int WT, bool LO>
__device__ __forceinline__ void fetch(typename Shape<WT, LO>::Tokens &b, const uint16_t *from, int64_t rest, int bytes) {
  using S = Shape<WT, LO>;
#pragma unroll
  for (int l = 0; l < S::kHalves; ++l) {
    const uint4 *v = reinterpret_cast<const uint4 *>(from + (l ? rest : 0));
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i)
#pragma unroll
      for (int u = 0; u < S::kPer / 8; ++u) {
        const uint4 *at = v + i * (S::kPer / 2) + u;  // 4 kPer columns of 2 bytes a step
        b[i][l][u] = i * 64 >= bytes ? make_uint4(0, 0, 0, 0) : LO ? *at : __ldg(at);
      }
  }
}

// acc[row tile][token tile][chain] += a stage's rows (32) x tokens (8 per tile)^T over this warp's columns, of which `bytes`
// of a row exist (and are zeros up to whole scales' columns).  With one
// tile its tokens are in b, with more they are fetched here.  8-bit weights: scales of the warp's 128 columns at s[0] (rows g)
// and s[1] (rows g + 8), the same for both row tiles; `odd`: what special() says of those rows.
template <int XT, int WT, int NT, bool LO>
__device__ __forceinline__ void consume(float (&acc)[kRowTiles][NT][kChains<NT, LO>][4], const uint8_t *stage, typename Shape<WT, LO>::Tokens &b,
                                        uint32_t (&odd)[kRowTiles][2], int bytes, const uint16_t *const (&from)[NT], const bool (&there)[NT], int64_t rest,
                                        const float *const (&s)[2], int warp, int lane) {
  using S = Shape<WT, LO>;
  constexpr bool k8 = S::k8;
  const int g = lane >> 2, q = lane & 3, at = warp * S::kSteps * 64;
  if (at >= bytes) return;
  float s0 = 0.f, s1 = 0.f;
  if constexpr (k8) s0 = __ldg(s[0]), s1 = __ldg(s[1]);
#pragma unroll
  for (int m = 0; m < kRowTiles; ++m) {
    uint32_t x0[S::kSteps][S::kPer / 2], x1[S::kSteps][S::kPer / 2];
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) {
      const uint8_t *row = stage + (m * 16 + g) * kPitch + at + i * 64 + q * 16;
      const uint4 w0 = *reinterpret_cast<const uint4 *>(row), w1 = *reinterpret_cast<const uint4 *>(row + 8 * kPitch);
      if constexpr (k8) {
        const uint32_t y0[4] = {w0.x, w0.y, w0.z, w0.w}, y1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x0[i][2 * j] = widen<XT, WT>(__byte_perm(y0[j], 0, 0x1404));
          x0[i][2 * j + 1] = widen<XT, WT>(__byte_perm(y0[j], 0, 0x3424));
          x1[i][2 * j] = widen<XT, WT>(__byte_perm(y1[j], 0, 0x1404));
          x1[i][2 * j + 1] = widen<XT, WT>(__byte_perm(y1[j], 0, 0x3424));
          odd[m][0] |= special<WT>(y0[j]);
          odd[m][1] |= special<WT>(y1[j]);
        }
      } else {
        x0[i][0] = w0.x, x0[i][1] = w0.y, x0[i][2] = w0.z, x0[i][3] = w0.w;
        x1[i][0] = w1.x, x1[i][1] = w1.y, x1[i][2] = w1.z, x1[i][3] = w1.w;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (NT > 1) fetch<WT, LO>(b, from[n], rest, there[n] ? bytes - at - q * 16 : 0);
      float sum[kChains<NT, LO>][4] = {};
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i)
#pragma unroll
        for (int u = 0; u < S::kPer / 8; ++u)
#pragma unroll
          for (int l = 0; l < S::kHalves; ++l) {
            float(&d)[4] = k8 ? sum[l % kChains<NT, LO>] : acc[m][n][l % kChains<NT, LO>];
            mma<XT>(d, x0[i][4 * u], x1[i][4 * u], x0[i][4 * u + 1], x1[i][4 * u + 1], b[i][l][u].x, b[i][l][u].y);
            mma<XT>(d, x0[i][4 * u + 2], x1[i][4 * u + 2], x0[i][4 * u + 3], x1[i][4 * u + 3], b[i][l][u].z, b[i][l][u].w);
          }
      if constexpr (k8) {
#pragma unroll
        for (int l = 0; l < kChains<NT, LO>; ++l) {
          acc[m][n][l][0] = fmaf(sum[l][0], s0, acc[m][n][l][0]);
          acc[m][n][l][1] = fmaf(sum[l][1], s0, acc[m][n][l][1]);
          acc[m][n][l][2] = fmaf(sum[l][2], s1, acc[m][n][l][2]);
          acc[m][n][l][3] = fmaf(sum[l][3], s1, acc[m][n][l][3]);
        }
      }
    }
  }
}

// The warps' sums of some tokens, side by side for whoever adds them: [warp][token][row]
struct Sums {
  float v[kWarps][kRoundTiles * kTile][kRows];
};

__device__ __forceinline__ float total(const Sums &s, int token, int row) {
  float v = s.v[0][token][row];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += s.v[w][token][row];
  return v;
}

__device__ __forceinline__ float activate(int act, float g) {
  if (act == GE_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  if (act == GE_RELU) return g > 0.f ? g : (g == g ? 0.f : g);
  return g / (1.f + expf(-g));
}

template <int XT>
__device__ __forceinline__ float round_trip(uint16_t v) {
  if constexpr (XT == GE_BF16) return __uint_as_float(uint32_t(v) << 16);
  else return __half2float(__ushort_as_half(v));
}

// A unit of work: `a` the active expert, `col` its first column of h or of y.
struct Unit {
  int a, col;
  bool up;
};

struct Shared {
  Choice c;
  Sums sums[kGroups][2];
  alignas(8) uint64_t full[kStages], empty[kStages];          // stages of the ring
  alignas(8) uint64_t taken[kQueue], ready[kQueue], out[kQueue], free[kQueue];  // a unit: named, its h there, written, forgotten
  uint32_t unit[kQueue], first[kQueue];  // which one, and its first stage's number
  Unit what[kQueue];
  alignas(8) uint64_t given[kJobs], added[kJobs];  // shares to be added
  int job[kJobs];                                  // of which columns
  volatile uint32_t quit;
  alignas(128) uint8_t ring[kStages][kRows * kPitch];
};

constexpr uint32_t kNoUnit = 0xffffffffu;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// zeros in their place
__device__ __forceinline__ void clear16(uint32_t dst, const void *any) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, 0;" ::"r"(dst), "l"(any) : "memory");
}

// this thread arrives on a barrier once its copies so far have landed
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t add_acq_rel(uint32_t *p, uint32_t by) {
  uint32_t v;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(v) : "l"(p), "r"(by) : "memory");
  return v;
}

__device__ __forceinline__ void add_release(uint32_t *p, uint32_t by) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(by) : "memory");
}

__device__ void give_up(const MoeParams &p, Shared &sh) {
  if (atomicCAS(p.status, 0u, static_cast<uint32_t>(GE_ERR_TIMEOUT)) == 0u) {
    p.status[1] = 0;
    p.status[2] = blockIdx.x;
  }
  atomicExch(&p.head->abort, 1u);
  sh.quit = 1u;
}

// Waits within a CTA: false where it gives up.  (They last as long as another CTA's h does, and four times the
// time a watcher waits for that at most.)
__device__ __forceinline__ bool wait_bar(const MoeParams &p, Shared &sh, const uint64_t &bar, uint32_t parity) {
  const uint32_t b = smem_u32(&bar);
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(b, parity, 20000u)) return true;
    if (sh.quit) return false;
    if (globaltimer_ns() - t0 > 4 * p.timeout_ns) {
      give_up(p, sh);
      return false;
    }
  }
}

struct Units {
  uint32_t up_cols, down_cols, n_up, n_all;
  __device__ __forceinline__ Units(const MoeParams &p, int n_active) {
    up_cols = (p.F + kUpCols - 1) / kUpCols;
    down_cols = (p.D + kDownCols - 1) / kDownCols;
    n_up = n_active * up_cols;
    n_all = n_up + n_active * down_cols;
  }
  __device__ __forceinline__ Unit of(uint32_t u) const {
    Unit r;
    r.up = u < n_up;
    const uint32_t v = r.up ? u : u - n_up, per = r.up ? up_cols : down_cols;
    r.a = v / per;
    r.col = (v - r.a * per) * (r.up ? kUpCols : kDownCols);
    return r;
  }
};

// A position in a ring of N.
template <int N>
struct Turn {
  int at;
  uint32_t phase;
  __device__ __forceinline__ explicit Turn(uint32_t number = 0) : at(number % N), phase(number / N & 1u) {}
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// How many units from number n on have passed `bars` (one at least: the first is waited for; each lane has looked at
// its own); 0 where that wait gave up.
__device__ __forceinline__ uint32_t units_there(const MoeParams &p, Shared &sh, const uint64_t (&bars)[kQueue], uint32_t n) {
  const uint32_t lane = threadIdx.x & 31;
  const Turn<kQueue> first(n), mine(n + lane);
  if (!__all_sync(0xffffffffu, wait_bar(p, sh, bars[first.at], first.phase))) return 0;
  const bool there = lane < kQueue && mbar_test_wait(smem_u32(&bars[mine.at]), mine.phase);
  return __ffs(~__ballot_sync(0xffffffffu, there)) - 1;
}

// The consumers' part of a unit with up to 8 NT tokens; false where a wait gave up.
template <int XT, int WT, int NT, bool UP>
__device__ bool do_unit(const MoeParams &p, Shared &sh, const Unit &u, Turn<kStages> st, int &round) {
  constexpr bool k8 = WT == GE_E4M3 || WT == GE_E5M2;
  constexpr int ws = k8 ? 1 : 2;
  const int warp = (threadIdx.x >> 5) % kWarps, group = threadIdx.x / (32 * kWarps), lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int thread = threadIdx.x % (32 * kWarps);
  const Choice &c = sh.c;
  const int e = c.active[u.a], n = c.count[u.a];
  const uint16_t *list = c.list + c.begin[u.a];
  using S = Shape<WT, !UP>;
  const int K = UP ? p.D : p.F;
  const int64_t rest = int64_t(p.T) * p.k * p.F;
  // Scales of rows: a unit's columns start at a multiple of 16 (of 32), so gate's lie in one block of rows, w_down's too;
  // up's start at F more, a multiple of 16.
  const float *scale[2] = {nullptr, nullptr};
  int64_t ld_s = 0;
  if constexpr (k8) {
    ld_s = ((UP ? 2 * p.F : p.D) + kBlock - 1) / kBlock;
    const float *f = (UP ? p.s_up : p.s_down) + int64_t(e) * ld_s * ((K + kBlock - 1) / kBlock) + warp * (kSegment / kWarps / kBlock) * ld_s;
    scale[0] = f + u.col / kBlock;
    scale[1] = f + (UP ? p.F + u.col : u.col) / kBlock;
  }
  const uint16_t *from[NT];
  bool there[NT];
  // this lane's first column of a stage
  const int mine = warp * S::kSteps * 64 + q * 16, col0 = mine / ws;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int at = i * kTile + g;
    there[i] = at < n;
    from[i] = (UP ? static_cast<const uint16_t *>(p.x) : p.h) + col0;
    if (there[i]) from[i] += UP ? int64_t(c.token[c.begin[u.a] + at]) * p.ldx : int64_t(list[at]) * p.F;
  }
  float acc[kRowTiles][NT][kChains<NT, !UP>][4] = {};
  uint32_t odd[kRowTiles][2] = {};
  for (int bytes = K * ws; bytes > 0; bytes -= kSegment) {
    typename S::Tokens b;  // (one tile's tokens are on their way while the stage is waited for)
    if constexpr (NT == 1) fetch<WT, !UP>(b, from[0], rest, there[0] ? bytes - mine : 0);
    if (!__all_sync(0xffffffffu, wait_bar(p, sh, sh.full[st.at], st.phase))) return false;
    consume<XT, WT, NT, !UP>(acc, sh.ring[st.at], b, odd, bytes, from, there, rest, scale, warp, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st.at]));
    st.next();
#pragma unroll
    for (int i = 0; i < NT; ++i) from[i] += kSegment / ws;
    if constexpr (k8) {
      scale[0] += kSegment / kBlock * ld_s;
      scale[1] += kSegment / kBlock * ld_s;
    }
  }
  if constexpr (k8) {
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        odd[m][i] |= __shfl_xor_sync(0xffffffffu, odd[m][i], 1);  // the lanes of a row
        odd[m][i] |= __shfl_xor_sync(0xffffffffu, odd[m][i], 2);
        if (odd[m][i]) {
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[m][n][0][2 * i] = acc[m][n][0][2 * i + 1] = NAN;
        }
      }
    }
  }
  // the warps' sums, 8 tokens at a time (a buffer's last readers have passed the barrier of the round between)
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    if (r * kTile >= n) break;
    Sums &s = sh.sums[group][round++ & 1];
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = acc[m][r][0][j];
        if constexpr (kChains<NT, !UP> == 2) v[j] += acc[m][r][1][j];
      }
      s.v[warp][2 * q][m * 16 + g] = v[0];
      s.v[warp][2 * q + 1][m * 16 + g] = v[1];
      s.v[warp][2 * q][m * 16 + g + 8] = v[2];
      s.v[warp][2 * q + 1][m * 16 + g + 8] = v[3];
    }
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "n"(32 * kWarps) : "memory");
    const int some = min(n - r * kTile, kTile);
    const uint16_t *of = list + r * kTile;
    if constexpr (UP) {
      for (int i = thread; i < some * kUpCols; i += 32 * kWarps) {
        const int token = i / kUpCols, col = i % kUpCols, row = (col >> 3) * 16 + (col & 7);
        if (u.col + col >= p.F) continue;
        const float v = activate(p.act, total(s, token, row)) * total(s, token, row + 8);
        const uint16_t hi = static_cast<uint16_t>(pack16(XT == GE_BF16, v, 0.f));
        const float left = v - round_trip<XT>(hi);
        uint16_t *h = p.h + int64_t(of[token]) * p.F + u.col + col;
        h[0] = hi;
        // (nothing is left of an infinity)
        h[rest] = isfinite(left) ? static_cast<uint16_t>(pack16(XT == GE_BF16, left, 0.f)) : 0;
      }
    } else {
      for (int i = thread; i < some * kDownCols; i += 32 * kWarps) {
        const int token = i / kDownCols, row = i % kDownCols;
        if (u.col + row < p.D) p.part[int64_t(of[token]) * p.D + u.col + row] = total(s, token, row) * c.weight[of[token]];
      }
    }
  }
  return true;
}

template <int XT, int WT, bool UP>
__device__ bool any_unit(const MoeParams &p, Shared &sh, const Unit &u, Turn<kStages> st, int &round) {
  const int n = sh.c.count[u.a];
  if (n <= kTile) return do_unit<XT, WT, 1, UP>(p, sh, u, st, round);
  if (n <= 2 * kTile) return do_unit<XT, WT, 2, UP>(p, sh, u, st, round);
  return do_unit<XT, WT, kMostTokens / kTile, UP>(p, sh, u, st, round);
}

// y's 32 columns of all tokens, shared by `adders` warps: a lane adds 8 columns of a token, in the order of its
// choice.  What that costs is the way to the shares and back: eight of two tokens are under way at a time.
template <int XT>
__device__ void add_shares(const MoeParams &p, int col, int adder, int adders) {
  constexpr int kTokens = 2, kAtOnce = 8;
  const int lane = threadIdx.x & 31, d0 = col + (lane & 3) * 8;
  if (d0 >= p.D) return;
#pragma unroll 1
  for (int t0 = adder * 8 + (lane >> 2); t0 < p.T; t0 += 8 * adders * kTokens) {
    float v[kTokens][8] = {};
#pragma unroll 1
    for (int j0 = 0; j0 < p.k; j0 += kAtOnce) {
      float4 x[kTokens][kAtOnce][2];
#pragma unroll
      for (int i = 0; i < kTokens; ++i)
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int t = t0 + i * 8 * adders;
          const bool on = t < p.T && j0 + j < p.k;
          const float4 *f = reinterpret_cast<const float4 *>(p.part + (int64_t(t) * p.k + j0 + j) * p.D + d0);
          x[i][j][0] = on ? __ldcg(f) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[i][j][1] = on ? __ldcg(f + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int i = 0; i < kTokens; ++i)
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const float4 a = x[i][j][0], c = x[i][j][1];
          v[i][0] += a.x, v[i][1] += a.y, v[i][2] += a.z, v[i][3] += a.w;
          v[i][4] += c.x, v[i][5] += c.y, v[i][6] += c.z, v[i][7] += c.w;
        }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int t = t0 + i * 8 * adders;
      if (t >= p.T) continue;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack16(XT == GE_BF16, v[i][2 * e], v[i][2 * e + 1]);
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + int64_t(t) * p.ldy + d0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int XT, int WT>
__global__ void __launch_bounds__(kThreads, 1) moe_experts_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  Shared &sh = *reinterpret_cast<Shared *>(smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u));
  constexpr int ws = WT == GE_E4M3 || WT == GE_E5M2 ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 32 * kProducers);
      mbar_init(smem_u32(&sh.empty[i]), kWarps);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(smem_u32(&sh.taken[i]), 1);
      mbar_init(smem_u32(&sh.ready[i]), 1);
      mbar_init(smem_u32(&sh.out[i]), kWarps);
      mbar_init(smem_u32(&sh.free[i]), 1);
    }
    for (int i = 0; i < kJobs; ++i) {
      mbar_init(smem_u32(&sh.given[i]), 1);
      mbar_init(smem_u32(&sh.added[i]), kProducers);
    }
    sh.quit = 0u;
    fence_mbarrier_init();
  }
  // (the ring is not in use yet: keys lie there)
  static_assert((kThreads / 32) * sizeof(ChoiceSpace) <= sizeof(sh.ring), "room for choices");
  ChoiceSpace &space = reinterpret_cast<ChoiceSpace *>(&sh.ring[0][0])[warp];
  griddep_wait();
  griddep_launch_dependents();
  if (p.expert) {
    for (int i = threadIdx.x; i < p.T * p.k; i += kThreads) {
      sh.c.expert[i] = __ldcg(p.expert + i);
      sh.c.weight[i] = __ldcg(p.share + i);
    }
  } else {
    for (int t = warp; t < p.T; t += kThreads / 32) choose(p, t, sh.c.expert, sh.c.weight, space, blockIdx.x == 0);
  }
  __syncthreads();
  make_lists(p, sh.c);
  const Units units(p, sh.c.n_active);
  Turn<kQueue> slot(0);
  Turn<kStages> st(0);

  if (warp >= kProducer && warp < kWatcher) {
    // The first producer takes tickets, one unit ahead of its need; the others learn of them as everyone does.
    const int part = warp - kProducer;
    static_assert(kProducers == kRowTiles, "a row tile each");
    uint32_t filled = 0, next = 0;
    if (part == 0 && lane == 0) next = atomicAdd(&p.head->ticket, 1u);
    bool ok = true;
    int ends = 0;
    while (ok) {
      uint32_t t;
      if (part == 0) {
        ok = __all_sync(0xffffffffu, wait_bar(p, sh, sh.free[slot.at], slot.phase ^ 1u));
        if (!ok) break;
        t = __shfl_sync(0xffffffffu, next, 0);
        if (t >= units.n_all) t = kNoUnit;
        else if (lane == 0) next = atomicAdd(&p.head->ticket, 1u);
        if (lane == 0) {
          sh.unit[slot.at] = t;
          sh.first[slot.at] = filled;
          if (t != kNoUnit) sh.what[slot.at] = units.of(t);
          mbar_arrive(smem_u32(&sh.taken[slot.at]));
        }
        __syncwarp();
      } else {
        ok = __all_sync(0xffffffffu, wait_bar(p, sh, sh.taken[slot.at], slot.phase));
        if (!ok) break;
        t = sh.unit[slot.at];
      }
      const Unit u = sh.what[slot.at];
      slot.next();
      if (t == kNoUnit) {
        if (++ends == kGroups) break;  // one for each group
        continue;
      }
      const int e = sh.c.active[u.a], K = u.up ? p.D : p.F;
      const uint8_t *w = static_cast<const uint8_t *>(u.up ? p.w_up : p.w_down);
      w += (int64_t(e) * (u.up ? 2 * int64_t(p.F) : int64_t(p.D)) + u.col) * K * ws + lane * 16;
      // this producer's 16 rows: of gate and of up eight each, or of w_down
      const int64_t pitch = int64_t(K) * ws, second = u.up ? int64_t(p.F) * pitch : 8 * pitch;
      const int rows = u.up ? (u.col + 8 * part < p.F ? 16 : 0) : min(16, p.D - u.col - 16 * part);
      w += (u.up ? 8 : 16) * part * pitch;
      for (int at = 0; at < K * ws; at += kSegment, w += kSegment) {
        ok = __all_sync(0xffffffffu, wait_bar(p, sh, sh.empty[st.at], st.phase ^ 1u));
        if (!ok) break;
        const int left = min(kSegment, K * ws - at), bytes = left - lane * 16;
        const uint32_t to = smem_u32(sh.ring[st.at]) + part * 16 * kPitch + lane * 16;
        if (rows == 16 && left == kSegment) {
          // (with as few instructions as can be: two warps issue all of an SM's copies)
          const uint8_t *row = w;
#pragma unroll
          for (int r = 0; r < 8; ++r, row += pitch) {
            const uint8_t *row8 = row + second;
#pragma unroll
            for (int j = 0; j < kSegment; j += 512) {
              copy16(to + r * kPitch + j, row + j);
              copy16(to + (r + 8) * kPitch + j, row8 + j);
            }
          }
        } else {
#pragma unroll 4
          for (int r = 0; r < rows; ++r)
#pragma unroll
            for (int j = 0; j < kSegment; j += 512)
              if (j < bytes) copy16(to + r * kPitch + j, w + (r & 7) * pitch + (r & 8 ? second : 0) + j);
        }
        if (left % 128 != 0) {  // up to a consumer's whole columns: fewer than 8 lanes' worth in each row
          const int end = left + (lane & 7) * 16;
          if (end < (left + 127) / 128 * 128)
            for (int r = lane >> 3; r < 16; r += 4) clear16(to + r * kPitch - lane * 16 + end, w);
        }
        arrive_after_copies(smem_u32(&sh.full[st.at]));
        st.next();
        ++filled;
      }
    }
    // (what is on its way lands before the CTA's shared memory is another's)
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (Turn<kJobs> job(0);; job.next()) {
      if (!__all_sync(0xffffffffu, wait_bar(p, sh, sh.given[job.at], job.phase))) break;
      const int col = sh.job[job.at];
      if (col < 0) break;
      add_shares<XT>(p, col, part, kProducers);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.added[job.at]));
    }
  } else if (warp == kWatcher) {
    // Lanes look after a unit each, as many as have been taken: one by one, a unit of few columns takes
    // less time than a look at another CTA's work does.  (Units that wait for nothing are passed on before any
    // wait: h may be theirs.)
    int ends = 0;
    for (uint32_t n = 0; ends < kGroups;) {
      const uint32_t some = units_there(p, sh, sh.taken, n);
      if (!some) break;
      const Turn<kQueue> at(n + lane);
      const uint32_t t = lane < some ? sh.unit[at.at] : 0;
      ends += __popc(__ballot_sync(0xffffffffu, t == kNoUnit));
      bool waits = lane < some && t != kNoUnit && t >= units.n_up;
      if (lane < some && !waits) mbar_arrive(smem_u32(&sh.ready[at.at]));
      const uint32_t *counter = p.done;
      uint32_t want = 0;
      if (waits) {
        const int a = sh.what[at.at].a;
        counter += sh.c.active[a];
        want = units.up_cols * sh.c.parts[a];
      }
      bool ok = true;
      const uint64_t t0 = __any_sync(0xffffffffu, waits) ? globaltimer_ns() : 0;
      while (true) {
        if (waits && load_acquire(counter) >= want) {
          mbar_arrive(smem_u32(&sh.ready[at.at]));
          waits = false;
        }
        if (!__any_sync(0xffffffffu, waits)) break;
        if (lane == 0) {
          if (load_acquire(&p.head->abort)) {
            sh.quit = 1u;
          } else if (globaltimer_ns() - t0 > p.timeout_ns) {
            give_up(p, sh);
          }
        }
        __syncwarp();
        ok = !sh.quit;
        if (!__all_sync(0xffffffffu, ok)) break;
        __nanosleep(64);
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      n += some;
    }
  } else if (warp == kFinisher) {
    // the same for units that have been written (and one fence for all of them)
    Turn<kJobs> job(0);
    auto give = [&](int col) {
      if (lane == 0) {
        sh.job[job.at] = col;
        mbar_arrive(smem_u32(&sh.given[job.at]));
      }
      __syncwarp();
      job.next();
    };
    int ends = 0;
    for (uint32_t n = 0; ends < kGroups;) {
      const uint32_t some = units_there(p, sh, sh.out, n);
      if (!some) break;
      const Turn<kQueue> at(n + lane);
      uint32_t t = 0;
      int col = 0;
      bool last = false;
      if (lane < some) {
        t = sh.unit[at.at];
        const Unit u = sh.what[at.at];
        col = u.col;
        mbar_arrive(smem_u32(&sh.free[at.at]));
        if (t != kNoUnit) {
          if (!u.up) last = add_acq_rel(&p.shares[u.col / kDownCols], 1u) == static_cast<uint32_t>(sh.c.n_active) - 1u;
          else if (t != 0 || !(p.debug_flags & GE_DEBUG_SKIP_FIRST_LOAD)) add_release(&p.done[sh.c.active[u.a]], 1u);
        }
      }
      for (uint32_t left = __ballot_sync(0xffffffffu, last); left; left &= left - 1) {
        const int its = __shfl_sync(0xffffffffu, col, __ffs(left) - 1);
        __syncwarp();  // (what that lane's counter has shown is there for all)
        // (not to wait for the producers, who may wait for units that this warp forgets)
        if (__all_sync(0xffffffffu, mbar_test_wait(smem_u32(&sh.added[job.at]), job.phase ^ 1u))) give(its);
        else add_shares<XT>(p, its, 0, 1);
      }
      ends += __popc(__ballot_sync(0xffffffffu, t == kNoUnit));
      n += some;
    }
    if (__all_sync(0xffffffffu, wait_bar(p, sh, sh.added[job.at], job.phase ^ 1u))) give(-1);
  } else {
    // group i takes units i, i + kGroups, ... of the CTA
    int round = 0;
    for (uint32_t n = warp / kWarps;; n += kGroups) {
      const Turn<kQueue> at(n);
      if (!__all_sync(0xffffffffu, wait_bar(p, sh, sh.ready[at.at], at.phase))) break;
      const uint32_t t = sh.unit[at.at];
      if (t != kNoUnit) {
        const Unit u = sh.what[at.at];
        const Turn<kStages> from(sh.first[at.at]);
        if (!(u.up ? any_unit<XT, WT, true>(p, sh, u, from, round) : any_unit<XT, WT, false>(p, sh, u, from, round))) break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.out[at.at]));
      if (t == kNoUnit) break;
    }
  }
}

constexpr int kMoeSmem = static_cast<int>(sizeof(Shared)) + 128;
static_assert(kMoeSmem <= 232448, "an SM's shared memory");

}  // namespace
}  // namespace ge
