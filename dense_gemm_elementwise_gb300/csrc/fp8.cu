// fp8.cu -- host side of the block-scaled 8-bit products (gemm_epi_fp8_*); the product is in fp8_kernel.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "fp8_kernel.cuh"
#include "gemm_epi.h"
#include "host.h"

using namespace ge;

namespace {

int64_t size_of(int t) { return t == GE_F32 ? 4 : 2; }

}  // namespace

struct gemm_epi_fp8_plan {
  int64_t M = 0, N = 0, K = 0;
  ge_fp8_desc d{};
  int sms = 0, cg = 1, cluster = 1, grid = 1, smem = 0;
  const void *fn = nullptr, *fn_add = nullptr;  // without and with C
  Fp8Params p{};
  bool few = false;  // fp8_few.cu's kernel
};

namespace {

int configure(gemm_epi_fp8_plan *pl, int max_smem) {
  Fp8Params &p = pl->p;
  const int64_t M = pl->M, N = pl->N;
  // Up to 16 rows of A have a kernel of their own (from memory, us: 8 x 2048 x 7168 5.3, the other one 9.4; 8 x 40000 x 4096 29.5
  // and 41.1; 16 x 2048 x 7168 6.2 and 9.6).  It wants blocks for its warps where there are many columns (1 x 100000 x 256 16.3 and
  // 14.1, x 512 16.7 and 17.3, but 1 x 20000 x 256 4.5 and 5.7), and with more than 8 rows its arithmetic shows
  // (16 x 100000 x 512 23.2 and 17.6, 12 x 16384 x 8192 33.0 and 27.0, but 16 x 8192 x 4096 10.7 and 11.6).
  // (What tests that a load which never comes is reported is the other kernel's: here nothing waits for another.)
  p.num_kb = static_cast<int32_t>(ceil_div(pl->K, kF8Block));
  const int64_t units = ceil_div(N, kF8FewUnit), slots = int64_t(pl->sms) * kF8FewPerSm;
  pl->few = M <= kF8FewRows && p.debug_flags == 0 &&
            (M <= 8 ? units <= 8 * slots || p.num_kb >= 4 : units <= 8 * slots && N * pl->K <= int64_t(1) << 26);
  if (pl->few) {
    const Fp8Few few = fp8_few(p.a_e5m2 != 0, p.b_e5m2 != 0, static_cast<int>(M));
    pl->fn = pl->fn_add = few.fn;
    pl->smem = few.smem;
    if (cudaFuncSetAttribute(pl->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, pl->smem) != cudaSuccess) {
      cudaGetLastError();
      return GE_ERR_CUDA;
    }
    pl->grid = static_cast<int>(std::min<int64_t>(units, pl->d.max_ctas > 0 ? pl->d.max_ctas : slots));
    return GE_OK;
  }
  const int ctas = pl->d.max_ctas > 0 ? std::min(pl->d.max_ctas, pl->sms) : pl->sms;
  pl->cg = M > 128 && ctas >= 2 && ceil_div(M, 256) * ceil_div(N, 256) > ctas / 4 ? 2 : 1;
  const int bm = 128 * pl->cg, bn = 128 * pl->cg, groups = ctas / pl->cg;
  const bool square = pl->d.b_block == GE_BLOCK_SQUARE;
  const bool turned = pl->d.ldd * size_of(pl->d.d) % 16 != 0;
  const auto pick = pl->cg == 2 ? fp8_kernel_cg2 : fp8_kernel_cg1;
  pl->fn = pick(square, false, turned);
  pl->fn_add = pick(square, true, turned);
  const int64_t num_m = ceil_div(M, bm), num_n = ceil_div(N, bn), tiles = num_m * num_n;
  if (tiles > (int64_t(1) << 31) / kF8MaxSlices) return GE_ERR_SHAPE;
  p.num_m_blk = static_cast<int32_t>(num_m);
  p.num_n_blk = static_cast<int32_t>(num_n);
  p.raster_group = num_m <= 16 ? static_cast<int32_t>(num_m) : 12;
  p.a_rows = pl->cg == 1 ? static_cast<int32_t>(std::min<int64_t>(128, round_up(M, 8))) : 128;
  const int stage = 128 * 128 + 128 * bn / pl->cg;
  const int fixed = 1024 + static_cast<int>(kF8BarBytes + fp8_scale_bytes(bn, square) + (turned ? kF8TurnBytes : 0u));
  p.stages = std::min(kMaxStages, (max_smem - fixed) / stage);
  if (p.stages < 2) return GE_ERR_SMEM;
  p.off_B = static_cast<uint32_t>(p.stages * 128 * 128);
  p.off_bar = static_cast<uint32_t>(p.stages * stage);
  p.off_turn = p.off_bar + kF8BarBytes + fp8_scale_bytes(bn, square);
  // the kernel's warps pass registers on, which have to be there
  pl->smem = max_smem;
  for (const void *fn : {pl->fn, pl->fn_add}) {
    cudaFuncAttributes fa;
    // (all of an SM's shared memory, so that its TMEM is this CTA's alone)
    if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess || fa.numRegs < kF8Regs ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) != cudaSuccess) {
      cudaGetLastError();
      return GE_ERR_CUDA;
    }
  }
  // Too few tiles for the GPU: their sums are split among the CTAs of clusters, all of which have to be there at once.
  // A slice more has to save a k-block (of about 0.3 us) for each slice: what it costs to join them.
  int slices = 1;
  for (int s = 2; pl->cg == 1 && s <= kF8MaxSlices && s <= p.num_kb && tiles * s <= groups; ++s) {
    if (ceil_div(p.num_kb, s) + s > ceil_div(p.num_kb, slices) + slices) continue;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(s);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * s));
    cfg.blockDim = dim3(kF8Threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(max_smem);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, pl->fn, &cfg) != cudaSuccess) {
      cudaGetLastError();
      continue;
    }
    if (clusters >= tiles) slices = s;
  }
  p.slices = slices;
  p.kb_split = static_cast<int32_t>(ceil_div(p.num_kb, slices));
  pl->cluster = pl->cg == 2 ? 2 : slices;
  pl->grid = static_cast<int>(std::min<int64_t>(groups, tiles * slices)) * pl->cg;
  return GE_OK;
}

}  // namespace

extern "C" {

int gemm_epi_fp8_plan_create(gemm_epi_fp8_plan **plan, int64_t M, int64_t N, int64_t K, const ge_fp8_desc *desc) {
  if (!plan) return GE_ERR_INVALID;
  *plan = nullptr;
  if (!desc) return GE_ERR_INVALID;
  for (int t : {desc->a, desc->b})
    if (t != GE_E4M3 && t != GE_E5M2) return GE_ERR_UNSUPPORTED;
  if (desc->d != GE_F16 && desc->d != GE_BF16 && desc->d != GE_F32) return GE_ERR_UNSUPPORTED;
  if ((desc->b_block != GE_BLOCK_ROW && desc->b_block != GE_BLOCK_SQUARE) || desc->timeout_ms < 0 || desc->max_ctas < 0 ||
      (desc->debug_flags & ~GE_DEBUG_SKIP_FIRST_LOAD) != 0 || desc->reserved != 0)
    return GE_ERR_INVALID;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  // (tiles' ends stay within 32 bits)
  if (M <= 0 || N <= 0 || K <= 0 || M > kMost - 256 || N > kMost - 256 || K > kMost - 256) return GE_ERR_SHAPE;
  ge_fp8_desc d = *desc;
  const struct { int64_t *ld; int64_t least; } pitch[] = {
      {&d.lda, K}, {&d.ldb, K}, {&d.ldd, N}, {&d.lds_a, M},
      {&d.lds_b, d.b_block == GE_BLOCK_SQUARE ? ceil_div(N, kF8Block) : N}};
  for (const auto &q : pitch) {
    if (*q.ld == 0) *q.ld = q.least;
    if (*q.ld < q.least || *q.ld > kMost) return GE_ERR_SHAPE;
  }
  if (d.lda % 16 != 0 || d.ldb % 16 != 0) return GE_ERR_MISALIGNED;
  gemm_epi_fp8_plan *pl = new (std::nothrow) gemm_epi_fp8_plan();
  if (!pl) return GE_ERR_INVALID;
  pl->M = M;
  pl->N = N;
  pl->K = K;
  pl->d = d;
  Fp8Params &p = pl->p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.lds_a = d.lds_a;
  p.lds_b = d.lds_b;
  p.ldd = d.ldd;
  p.dt = d.d;
  p.a_e5m2 = d.a == GE_E5M2;
  p.b_e5m2 = d.b == GE_E5M2;
  p.debug_flags = d.debug_flags;
  p.timeout_ns = uint64_t(d.timeout_ms > 0 ? d.timeout_ms : 1000) * 1000000u;
  int dev = 0, max_smem = 0;
  int st = current_device(&dev, &pl->sms, &max_smem);
  if (st == GE_OK) {
    p.status = status_block();
    if (!p.status) st = GE_ERR_CUDA;
  }
  if (st == GE_OK) st = configure(pl, max_smem);
  if (st != GE_OK) {
    delete pl;
    return st;
  }
  *plan = pl;
  return GE_OK;
}

void gemm_epi_fp8_plan_destroy(gemm_epi_fp8_plan *plan) { delete plan; }

// (sums that are split are joined in shared memory)
size_t gemm_epi_fp8_workspace_bytes(const gemm_epi_fp8_plan *) { return 0; }

int gemm_epi_fp8_run(gemm_epi_fp8_plan *pl, const void *A, const float *scale_a, const void *B, const float *scale_b,
                     const void *C, void *D, void *workspace, size_t workspace_bytes, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  if (!A || !B || !D || !scale_a || !scale_b) return GE_ERR_MISSING_ARG;
  for (const void *q : {A, B, C, static_cast<const void *>(D)})
    if (!is_aligned16(q)) return GE_ERR_MISALIGNED;
  for (const float *q : {scale_a, scale_b})
    if ((reinterpret_cast<uintptr_t>(q) & 3u) != 0) return GE_ERR_MISALIGNED;
  if (!is_aligned16(workspace)) return GE_ERR_MISALIGNED;
  if (workspace_bytes < gemm_epi_fp8_workspace_bytes(pl)) return GE_ERR_WORKSPACE;
  Fp8Params p = pl->p;
  p.sa = scale_a;
  p.sb = scale_b;
  p.c = C;
  p.d = D;
  if (pl->few) {
    int32_t K = static_cast<int32_t>(pl->K);
    bool square = pl->d.b_block == GE_BLOCK_SQUARE;
    void *args[] = {&p, &A, &B, &pl->d.lda, &pl->d.ldb, &K, &square};
    return launch_pdl(pl->fn, dim3(static_cast<unsigned>(pl->grid)), dim3(kF8FewThreads), pl->smem, args, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GE_OK
               : GE_ERR_CUDA;
  }
  if (!encode_rows(&p.tmA, GE_E4M3, A, pl->K, pl->M, 1, pl->d.lda, pl->d.lda * pl->M, kF8Block, p.a_rows) ||
      !encode_rows(&p.tmB, GE_E4M3, B, pl->K, pl->N, 1, pl->d.ldb, pl->d.ldb * pl->N, kF8Block, 128))
    return GE_ERR_CUDA;
  // (bases are whole 16 bytes)
  const int64_t pitch = p.ldd * size_of(p.dt);
  p.vec = pitch % 32 != 0 || ((reinterpret_cast<uintptr_t>(C) | reinterpret_cast<uintptr_t>(D)) & 31u) != 0 ? 1 : 2;
  void *args[] = {&p};
  return launch_pdl(C ? pl->fn_add : pl->fn, dim3(static_cast<unsigned>(pl->grid)), dim3(kF8Threads), pl->smem, args, static_cast<cudaStream_t>(stream),
                    pl->cluster) == cudaSuccess ? GE_OK : GE_ERR_CUDA;
}

}  // extern "C"
