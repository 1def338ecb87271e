// fp8.cu -- host side of the block-scaled 8-bit products (gemm_epi_fp8_*), and the kernel that
// joins the slices of a split sum; the product is in fp8_kernel.cuh.
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

struct JoinParams {
  Fp8Params p;  // c, d, part, sizes
};

// The slices of 8 columns of a row, added in order.
__global__ void __launch_bounds__(256) fp8_join_kernel(const __grid_constant__ JoinParams q) {
  const Fp8Params &p = q.p;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t groups = p.ld_part / 8, all = groups * p.M;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t m = i / groups, n = (i - m * groups) * 8;
    if (n >= p.N) continue;
    float v[8] = {};
    const float4 *s = reinterpret_cast<const float4 *>(p.part + m * p.ld_part + n);
#pragma unroll 4
    for (int z = 0; z < p.slices; ++z) {
      const float4 a = __ldcg(s), b = __ldcg(s + 1);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      s += int64_t(p.M) * p.ld_part / 4;
    }
    const int64_t at = m * p.ldd + n;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < p.N) store_one(p.d, at + e, p.dt, v[e] + (p.c ? load_one(p.c, at + e, p.dt) : 0.f));
  }
}

int64_t size_of(int t) { return t == GE_F32 ? 4 : 2; }

}  // namespace

struct gemm_epi_fp8_plan {
  int64_t M = 0, N = 0, K = 0;
  ge_fp8_desc d{};
  int sms = 0, cg = 1, grid = 1, smem = 0;
  const void *fn = nullptr;
  Fp8Params p{};
};

namespace {

int configure(gemm_epi_fp8_plan *pl, int max_smem) {
  Fp8Params &p = pl->p;
  const int64_t M = pl->M, N = pl->N;
  const int ctas = pl->d.max_ctas > 0 ? std::min(pl->d.max_ctas, pl->sms) : pl->sms;
  pl->cg = M > 128 && ctas >= 2 && ceil_div(M, 256) * ceil_div(N, 256) > ctas / 4 ? 2 : 1;
  const int bm = 128 * pl->cg, bn = 128 * pl->cg, units = ctas / pl->cg;
  const bool square = pl->d.b_block == GE_BLOCK_SQUARE;
  pl->fn = pl->cg == 2 ? fp8_kernel_cg2(square) : fp8_kernel_cg1(square);
  const int64_t num_m = ceil_div(M, bm), num_n = ceil_div(N, bn), tiles = num_m * num_n;
  p.num_kb = static_cast<int32_t>(ceil_div(pl->K, kF8Block));
  // too few tiles for the GPU: their sums are split
  int64_t slices = 1;
  if (tiles < units) slices = std::min<int64_t>(units / tiles, p.num_kb);
  p.kb_split = static_cast<int32_t>(ceil_div(p.num_kb, slices));
  slices = ceil_div(p.num_kb, p.kb_split);
  if (tiles * slices > (int64_t(1) << 31) - 1) return GE_ERR_SHAPE;
  p.slices = static_cast<int32_t>(slices);
  p.ld_part = round_up(N, bn);
  p.num_m_blk = static_cast<int32_t>(num_m);
  p.num_n_blk = static_cast<int32_t>(num_n);
  p.raster_group = num_m <= 16 ? static_cast<int32_t>(num_m) : 12;
  p.a_rows = pl->cg == 1 ? static_cast<int32_t>(std::min<int64_t>(128, round_up(M, 8))) : 128;
  const int stage = 128 * 128 + 128 * bn / pl->cg;
  const int fixed = 1024 + static_cast<int>(kF8BarBytes + fp8_scale_bytes(bn, square));
  p.stages = std::min(kMaxStages, (max_smem - fixed) / stage);
  if (p.stages < 2) return GE_ERR_SMEM;
  p.off_B = static_cast<uint32_t>(p.stages * 128 * 128);
  p.off_bar = static_cast<uint32_t>(p.stages * stage);
  // the kernel's warps pass registers on, which have to be there
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, pl->fn) != cudaSuccess || fa.numRegs < kF8Regs) {
    cudaGetLastError();
    return GE_ERR_CUDA;
  }
  // all of an SM's shared memory, so that its TMEM is this CTA's alone
  pl->smem = max_smem;
  if (cudaFuncSetAttribute(pl->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) != cudaSuccess) {
    cudaGetLastError();
    return GE_ERR_CUDA;
  }
  pl->grid = static_cast<int>(std::min<int64_t>(units, tiles * slices)) * pl->cg;
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

size_t gemm_epi_fp8_workspace_bytes(const gemm_epi_fp8_plan *pl) {
  if (!pl || pl->p.slices == 1) return 0;
  // (16 more, to start on a whole 32 bytes)
  return 16 + sizeof(float) * static_cast<size_t>(pl->p.slices) * static_cast<size_t>(pl->M) * static_cast<size_t>(pl->p.ld_part);
}

int gemm_epi_fp8_run(gemm_epi_fp8_plan *pl, const void *A, const float *scale_a, const void *B, const float *scale_b,
                     const void *C, void *D, void *workspace, size_t workspace_bytes, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  if (!A || !B || !D || !scale_a || !scale_b) return GE_ERR_MISSING_ARG;
  for (const void *q : {A, B, C, static_cast<const void *>(D)})
    if (!is_aligned16(q)) return GE_ERR_MISALIGNED;
  for (const float *q : {scale_a, scale_b})
    if ((reinterpret_cast<uintptr_t>(q) & 3u) != 0) return GE_ERR_MISALIGNED;
  const size_t need = gemm_epi_fp8_workspace_bytes(pl);
  if (need && (!workspace || workspace_bytes < need)) return GE_ERR_WORKSPACE;
  if (need && !is_aligned16(workspace)) return GE_ERR_MISALIGNED;
  Fp8Params p = pl->p;
  if (!encode_rows(&p.tmA, GE_E4M3, A, pl->K, pl->M, 1, pl->d.lda, pl->d.lda * pl->M, kF8Block, p.a_rows) ||
      !encode_rows(&p.tmB, GE_E4M3, B, pl->K, pl->N, 1, pl->d.ldb, pl->d.ldb * pl->N, kF8Block, 128))
    return GE_ERR_CUDA;
  p.sa = scale_a;
  p.sb = scale_b;
  p.c = C;
  p.d = D;
  p.part = need ? reinterpret_cast<float *>(round_up(static_cast<int64_t>(reinterpret_cast<uintptr_t>(workspace)), 32)) : nullptr;
  auto rows32 = [&](const void *q) { return !q || ((reinterpret_cast<uintptr_t>(q) | static_cast<uintptr_t>(p.ldd * size_of(p.dt))) & 31u) == 0; };
  p.vec = rows32(C) && rows32(D);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void *args[] = {&p};
  if (launch_pdl(pl->fn, dim3(pl->grid), dim3(kF8Threads), pl->smem, args, s, pl->cg) != cudaSuccess) return GE_ERR_CUDA;
  if (p.slices == 1) return GE_OK;
  JoinParams q;
  q.p = p;
  const int64_t threads = p.ld_part / 8 * pl->M;
  void *jargs[] = {&q};
  return launch_pdl(reinterpret_cast<const void *>(fp8_join_kernel), dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(threads, 256), pl->sms * 8))),
                    dim3(256), 0, jargs, s) == cudaSuccess ? GE_OK : GE_ERR_CUDA;
}

}  // extern "C"
