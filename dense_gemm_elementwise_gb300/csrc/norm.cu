// norm.cu -- host side of the norms around a block (gemm_epi_norm_*), and the
// kernel that adds the partial sums over rows; the rest is in norm_kernel.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "gemm_epi.h"
#include "host.h"
#include "norm_kernel.cuh"

using namespace ge;

namespace {

// Adds the units' partial rows.  grid.y 0: dw_pre and dw_post; grid.y 1 + g: the
// gate of group g (units that hold part of one group).  A thread adds every 32nd unit
// of four columns, then the 32 sums of a column are added in order.  It is bound by the
// latency of its loads: 16 bytes at a time and four units ahead.
struct SumParams {
  const float *part_pre, *part_post;
  int64_t ld_part;
  const void *gate, *w_post;
  void *dgate, *dw_post, *dw_pre;
  float alpha;
  int32_t D, wt, units, units_per_group;
};

constexpr int kSumCols = 32, kSumQuads = kSumCols / 4, kSumLanes = 32;

__global__ void __launch_bounds__(kSumQuads *kSumLanes) norm_sum_kernel(const __grid_constant__ SumParams p) {
  __shared__ float part[2][kSumLanes][kSumCols + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int quad = threadIdx.x % kSumQuads, lane = threadIdx.x / kSumQuads;
  const int col = blockIdx.x * kSumCols + quad * 4;
  // rows of partial sums are padded to whole quads of columns
  const bool on = col < p.D;
  float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [](float (&s)[4], const float4 &v) { s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w; };
  if (blockIdx.y == 0) {
    const bool pre = p.dw_pre != nullptr, post = p.dw_post != nullptr;
    const bool gated = p.gate && p.units_per_group;  // units of whole groups have their gates in the sum already
#pragma unroll 4
    for (int u = lane; u < (on ? p.units : 0); u += kSumLanes) {
      const int64_t at = int64_t(u) * p.ld_part + col;
      if (pre) add(a, *reinterpret_cast<const float4 *>(p.part_pre + at));
      if (post) {
        float4 q = *reinterpret_cast<const float4 *>(p.part_post + at);
        if (gated) {
          const int64_t g = int64_t(u / p.units_per_group) * p.D;
          q.x *= getw(p.wt, p.gate, g + col);
          q.y *= getw(p.wt, p.gate, g + min(col + 1, p.D - 1));
          q.z *= getw(p.wt, p.gate, g + min(col + 2, p.D - 1));
          q.w *= getw(p.wt, p.gate, g + min(col + 3, p.D - 1));
        }
        add(b, q);
      }
    }
  } else {
    const int64_t first = int64_t(blockIdx.y - 1) * p.units_per_group;
#pragma unroll 4
    for (int s = lane; s < (on ? p.units_per_group : 0); s += kSumLanes)
      add(a, *reinterpret_cast<const float4 *>(p.part_post + (first + s) * p.ld_part + col));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    part[0][lane][quad * 4 + i] = a[i];
    part[1][lane][quad * 4 + i] = b[i];
  }
  __syncthreads();
  if (threadIdx.x >= 2 * kSumCols) return;
  const int which = threadIdx.x / kSumCols, c = threadIdx.x % kSumCols, at = blockIdx.x * kSumCols + c;
  if (at >= p.D) return;
  float s = 0.f;
#pragma unroll
  for (int l = 0; l < kSumLanes; ++l) s += part[which][l][c];
  if (blockIdx.y == 0) {
    if (which == 0 && p.dw_pre) putw(p.wt, p.dw_pre, at, s);
    if (which == 1 && p.dw_post) putw(p.wt, p.dw_post, at, p.alpha * s);
  } else if (which == 0) {
    const float w = p.w_post ? getw(p.wt, p.w_post, at) : 1.f;
    putw(p.wt, p.dgate, int64_t(blockIdx.y - 1) * p.D + at, p.alpha * w * s);
  }
}

enum NormPass { PASS_RUN = 0, PASS_GRAD = 1, PASS_GRAD_WHOLE = 2 };

const void *pick_kernel(int dt, int nv, int threads, int rows, bool even, int pass) {
  if (rows == ROWS_16)
    return pass == PASS_RUN    ? norm_kernel_run(dt, nv)
           : pass == PASS_GRAD ? norm_kernel_grad(dt, nv)
                               : norm_kernel_grad_whole(dt, nv);
  if (rows == ROWS_SMALL)
    return pass == PASS_RUN    ? norm_kernel_run_small(dt, nv, threads, even)
           : pass == PASS_GRAD ? norm_kernel_grad_small(dt, nv, threads, even)
                               : norm_kernel_grad_whole_small(dt, nv, threads, even);
  return pass == PASS_RUN    ? norm_kernel_run_odd(dt, nv, threads)
         : pass == PASS_GRAD ? norm_kernel_grad_odd(dt, nv, threads)
                             : norm_kernel_grad_whole_odd(dt, nv, threads);
}

bool valid_type(int t) { return t == GE_F16 || t == GE_BF16 || t == GE_F32; }
int64_t size_of(int t) { return t == GE_F32 ? 4 : 2; }

// How a row is shared out: chunks of 8 columns per thread, threads per row,
// rows of the ring.
struct RowShape {
  const void *fn = nullptr;
  int nv = 1, row_threads = 32, threads = 32, grid = 1, ahead = 1, smem = 0;
};

cudaError_t launch(const void *fn, dim3 grid, dim3 block, int smem, void *params, cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void *args[] = {params};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

struct gemm_epi_norm_plan {
  int64_t T = 0, D = 0;
  ge_norm_desc d{};
  int sms = 0;
  bool vec = false, even = false;
  RowShape fwd, bwd;
  NormParams p{};
};

namespace {

int shape_of(const gemm_epi_norm_plan *pl, int pass, int max_smem, RowShape *out) {
  const int chunks = static_cast<int>(ceil_div(pl->D, kChunk));
  const int tensors = pass == PASS_RUN ? 2 : 4;
  RowShape r;
  // Rows of whole 16-byte units: two chunks per thread spread the cost of the row's sums (shuffles, a
  // barrier) over 16 columns, but rows too few to fill the GPU, and rows of
  // up to a warp's chunks, take one; what 512 threads cannot hold so takes four.
  // Rows moved 4 or 8 bytes at a time: two in CTAs of over 512 columns' chunks only (with two,
  // the gradients of 8000 x 2050 fp32 take 193 us, not 107), and above 1024 chunks CTAs of up to
  // 1024 threads (500 x 12346 bf16 35 us and its gradients 85, with four chunks 33 and 97).
  // Odd rows of 16-bit elements: one up to 1024 threads, since each element has a register
  // of its own on its way.
  const int rows_by = pl->vec ? ROWS_16 : pl->even || pl->d.x == GE_F32 ? ROWS_SMALL : ROWS_ODD;
  const int64_t few = 4 * int64_t(pl->sms);
  if (rows_by == ROWS_16)
    r.nv = chunks <= 32 || (pl->T <= few && chunks <= kVecThreads) ? 1 : (chunks <= 2 * kVecThreads ? 2 : 4);
  else
    r.nv = chunks <= (rows_by == ROWS_SMALL ? kVecThreads : kMaxThreads) ? 1 : 2;
  const int want = static_cast<int>(ceil_div(chunks, r.nv));
  r.row_threads = static_cast<int>(round_up(want, 32));
  if (want < 32) {  // rows share warps
    r.row_threads = 1;
    while (r.row_threads < want) r.row_threads *= 2;
  }
  // several short rows to a CTA of up to 256 threads, once there are enough of them
  // for every SM; whole warps
  int64_t cta_rows = std::max(1, 256 / r.row_threads);
  cta_rows = std::min<int64_t>(cta_rows, std::max<int64_t>(ceil_div(pl->T, few), r.row_threads < 32 ? 32 / r.row_threads : 1));
  if (r.row_threads < 32) cta_rows = round_up(cta_rows, 32 / r.row_threads);
  r.threads = r.row_threads * static_cast<int>(cta_rows);
  const int rows = r.threads / r.row_threads;
  r.fn = pick_kernel(pl->d.x, r.nv, r.threads, rows_by, pl->even, pass);
  // shared memory: sums, factors in fp32, and as many rows of the ring as let two CTAs
  // (three of the forward pass) share an SM, one at least: 512 threads' fp32 rows and
  // factors take 224 KiB
  const int fixed = kSumBytes + r.threads * r.nv * (pass == PASS_GRAD_WHOLE ? 6 : 4) * 16;
  const int per_row = r.threads * r.nv * tensors * static_cast<int>(size_of(pl->d.x)) * kChunk;
  r.ahead = 1;
  r.smem = fixed;
  if ((rows_by == ROWS_16 && r.nv < 4) || (rows_by == ROWS_SMALL && r.threads <= kVecThreads)) {
    const int room = max_smem / std::max(1, std::min(pass == PASS_RUN ? 3 : 2, 768 / r.threads));
    while (r.ahead < kMaxAhead && fixed + (r.ahead + 1) * per_row <= room) ++r.ahead;
    r.smem = fixed + r.ahead * per_row;
  }
  if (r.smem > max_smem) return GE_ERR_SMEM;
  int per_sm = 0;
  // the kernel's limit, which all of its plans share: the most there is, not what this one needs
  if (cudaFuncSetAttribute(r.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, r.fn, r.threads, static_cast<size_t>(r.smem)) !=
          cudaSuccess ||
      per_sm < 1) {
    cudaGetLastError();
    return GE_ERR_CUDA;
  }
  r.grid = static_cast<int>(std::min<int64_t>(ceil_div(pl->T, rows), int64_t(pl->sms) * per_sm));
  *out = r;
  return GE_OK;
}

void set_shape(NormParams *p, const RowShape &r) {
  p->row_threads = r.row_threads;
  p->ahead = r.ahead;
}

// Units of the gradient pass: CTAs, whose lanes hold whole gate groups (`whole` holds that
// kernel's shape) or which stay inside one.  Of the ways to cut groups up or put them together, the
// one whose waves of CTAs take the fewest rows one after another, where a CTA costs as much
// as kStart rows besides its own: its start, its partial sums and their adding up. (Groups
// of 12 put together to just under a wave's share, 328 units for 304 CTAs: 15735 x 1808 f16 in
// 159 us, rounded up 136.)
bool share_rows(gemm_epi_norm_plan *pl, const RowShape &whole) {
  constexpr int64_t kStart = 6;
  NormParams &p = pl->p;
  const RowShape &part = pl->bwd;
  const int64_t lanes = part.threads / part.row_threads;
  const int64_t rpg = pl->d.rows_per_gate ? std::min<int64_t>(pl->d.rows_per_gate, pl->T) : pl->T;
  const int64_t groups = ceil_div(pl->T, rpg);
  int64_t best = INT64_MAX;
  auto offer = [&](int64_t per_lane, int64_t per_group, int64_t units, int64_t grid) {
    if (per_lane * lanes > INT32_MAX || units > INT32_MAX) return;
    const int64_t cost = ceil_div(units, grid) * (per_lane + kStart);
    if (cost >= best) return;
    best = cost;
    p.rows_per_lane = static_cast<int32_t>(per_lane);
    p.rows_per_unit = static_cast<int32_t>(per_lane * lanes);
    p.units_per_group = static_cast<int32_t>(per_group);
    p.units = static_cast<int32_t>(units);
  };
  if (pl->d.rows_per_gate)
    for (int64_t waves = 1; waves <= 4; ++waves) {
      const int64_t g = ceil_div(ceil_div(ceil_div(pl->T, waves * whole.grid), lanes), rpg);
      offer(g * rpg, 0, ceil_div(pl->T, g * rpg * lanes), whole.grid);
    }
  if (groups < 65535)  // one row of norm_sum_kernel's grid each
    for (int64_t u = 1, most = ceil_div(rpg, ceil_div(pl->T, part.grid)) + 3; u <= most; ++u) {
      const int64_t per_lane = ceil_div(ceil_div(rpg, u), lanes);
      const int64_t per_group = ceil_div(rpg, per_lane * lanes);
      offer(per_lane, per_group, groups * per_group, part.grid);
    }
  return p.units_per_group == 0;
}

int check_ptr(const void *p) { return !p ? GE_ERR_MISSING_ARG : (is_aligned16(p) ? GE_OK : GE_ERR_MISALIGNED); }
int check_opt(const void *p) { return !p || is_aligned16(p) ? GE_OK : GE_ERR_MISALIGNED; }

// gate, w_post and w_pre as both passes take them
int check_block(const gemm_epi_norm_plan *pl, const void *b, const void *gate, const void *w_post,
                const void *w_pre) {
  for (const void *q : {b, gate, w_post, w_pre})
    if (check_opt(q) != GE_OK) return GE_ERR_MISALIGNED;
  if (!b) return gate || w_post ? GE_ERR_INVALID : GE_OK;
  if (pl->d.rows_per_gate && !gate) return GE_ERR_MISSING_ARG;
  if (!pl->d.rows_per_gate && gate) return GE_ERR_INVALID;
  if (pl->d.post == GE_NORM_NONE && w_post) return GE_ERR_INVALID;
  return GE_OK;
}

}  // namespace

extern "C" {

int gemm_epi_norm_plan_create(gemm_epi_norm_plan **plan, int64_t T, int64_t D, const ge_norm_desc *desc) {
  if (!plan) return GE_ERR_INVALID;
  *plan = nullptr;
  if (!desc) return GE_ERR_INVALID;
  if (!valid_type(desc->x) || !valid_type(desc->w)) return GE_ERR_UNSUPPORTED;
  if (desc->pre != GE_NORM_RMS && desc->pre != GE_NORM_LAYER) return GE_ERR_INVALID;
  if (desc->post < GE_NORM_NONE || desc->post > GE_NORM_LAYER) return GE_ERR_INVALID;
  if (!(desc->eps_pre >= 0.f) || !(desc->eps_post >= 0.f) || !std::isfinite(desc->eps_pre) ||
      !std::isfinite(desc->eps_post) || !std::isfinite(desc->alpha) || desc->reserved != 0 ||
      desc->rows_per_gate < 0)
    return GE_ERR_INVALID;
  if (T <= 0 || D <= 0 || D > GE_NORM_MAX_D || T > (int64_t(1) << 31) - 1) return GE_ERR_SHAPE;
  ge_norm_desc d = *desc;
  for (int64_t *ld : {&d.ldx, &d.ldb, &d.ldy, &d.ldh}) {
    if (*ld == 0) *ld = D;
    if (*ld < D || *ld > (int64_t(1) << 31) - 1) return GE_ERR_SHAPE;
  }
  gemm_epi_norm_plan *pl = new (std::nothrow) gemm_epi_norm_plan();
  if (!pl) return GE_ERR_INVALID;
  pl->T = T;
  pl->D = D;
  pl->d = d;
  const int64_t es = size_of(d.x);
  pl->vec = true;
  pl->even = true;
  for (int64_t ld : {d.ldx, d.ldb, d.ldy, d.ldh}) {
    pl->vec = pl->vec && (ld * es) % 16 == 0;
    pl->even = pl->even && ld % 2 == 0;
  }
  int dev = 0, smem = 0;
  int st = current_device(&dev, &pl->sms, &smem);
  if (st == GE_OK) st = shape_of(pl, PASS_RUN, smem, &pl->fwd);
  if (st == GE_OK) st = shape_of(pl, PASS_GRAD, smem, &pl->bwd);
  if (st != GE_OK) {
    delete pl;
    return st;
  }
  NormParams &p = pl->p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  p.ldx = d.ldx;
  p.ldb = d.ldb;
  p.ldy = d.ldy;
  p.ldh = d.ldh;
  // without a gate, one group of all rows
  p.rows_per_gate = d.rows_per_gate ? std::min<int64_t>(d.rows_per_gate, T) : T;
  p.T = static_cast<int32_t>(T);
  p.D = static_cast<int32_t>(D);
  p.wt = d.w;
  p.w_vec = (D * size_of(d.w)) % 16 == 0;
  p.ld_part = round_up(D, 8);
  p.pre = d.pre;
  p.post = d.post;
  p.eps_pre = d.eps_pre;
  p.eps_post = d.eps_post;
  p.alpha = d.alpha;
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(D));
  RowShape whole;
  st = shape_of(pl, PASS_GRAD_WHOLE, smem, &whole);
  if (st != GE_OK) {
    delete pl;
    return st;
  }
  if (share_rows(pl, whole)) pl->bwd = whole;
  *plan = pl;
  return GE_OK;
}

void gemm_epi_norm_plan_destroy(gemm_epi_norm_plan *plan) { delete plan; }

size_t gemm_epi_norm_workspace_bytes(const gemm_epi_norm_plan *pl) {
  if (!pl) return 0;
  return 2u * sizeof(float) * static_cast<size_t>(pl->p.units) * static_cast<size_t>(pl->p.ld_part);
}

int gemm_epi_norm_run(gemm_epi_norm_plan *pl, const void *x, const void *b, const void *gate,
                      const void *w_post, const void *w_pre, void *y, void *h, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  int st = check_ptr(x);
  if (st == GE_OK) st = check_block(pl, b, gate, w_post, w_pre);
  if (st != GE_OK) return st;
  if (!y && !h) return GE_ERR_MISSING_ARG;
  if (check_opt(y) != GE_OK || check_opt(h) != GE_OK) return GE_ERR_MISALIGNED;
  const ge_norm_desc &d = pl->d;
  // in place: a row is read before it is written only where the rows coincide
  if (y && y == h) return GE_ERR_INVALID;
  if ((y == x && d.ldy != d.ldx) || (b && y == b && d.ldy != d.ldb) || (h == x && d.ldh != d.ldx) ||
      (b && h == b && d.ldh != d.ldb))
    return GE_ERR_INVALID;
  NormParams p = pl->p;
  p.x = x;
  p.b = b;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.y = y;
  p.h = h;
  set_shape(&p, pl->fwd);
  const int64_t rows = pl->fwd.threads / pl->fwd.row_threads;
  p.rows_per_unit = b && gate && p.rows_per_gate < pl->T
                        ? static_cast<int32_t>(ceil_div(ceil_div(pl->T, rows), pl->fwd.grid) * rows) : 0;
  const cudaError_t e = launch(pl->fwd.fn, dim3(pl->fwd.grid), dim3(pl->fwd.threads), pl->fwd.smem, &p,
                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GE_OK : GE_ERR_CUDA;
}

int gemm_epi_norm_grad(gemm_epi_norm_plan *pl, const void *dy, const void *dh, const void *y,
                       const void *b, const void *gate, const void *w_post, const void *w_pre,
                       void *dx, void *db, void *dgate, void *dw_post, void *dw_pre,
                       void *workspace, size_t workspace_bytes, void *stream) {
  if (!pl) return GE_ERR_INVALID;
  for (const void *q : {dh, y, static_cast<const void *>(dx)}) {
    const int st = check_ptr(q);
    if (st != GE_OK) return st;
  }
  int st = check_block(pl, b, gate, w_post, w_pre);
  if (st != GE_OK) return st;
  for (const void *q : {dy, static_cast<const void *>(db), static_cast<const void *>(dgate),
                        static_cast<const void *>(dw_post), static_cast<const void *>(dw_pre)})
    if (check_opt(q) != GE_OK) return GE_ERR_MISALIGNED;
  // a gradient of something that takes no part
  if ((!b && (db || dgate || dw_post)) || (!gate && dgate) || (!w_post && dw_post) || (!w_pre && dw_pre))
    return GE_ERR_INVALID;
  const ge_norm_desc &d = pl->d;
  // in place, as in the forward pass
  if (dx == db) return GE_ERR_INVALID;
  const struct { const void *p; int64_t ld; } in[] = {{dy, d.ldy}, {dh, d.ldh}, {y, d.ldy}, {b, d.ldb}};
  for (const auto &q : in)
    if ((dx == q.p && d.ldx != q.ld) || (db && db == q.p && d.ldb != q.ld)) return GE_ERR_INVALID;
  if (!workspace || !is_aligned16(workspace) || workspace_bytes < gemm_epi_norm_workspace_bytes(pl))
    return GE_ERR_WORKSPACE;
  NormParams p = pl->p;
  p.dy = dy;
  p.dh = dh;
  p.yin = y;
  p.b = b;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.dx = dx;
  p.db = db;
  p.dgate = dgate;
  set_shape(&p, pl->bwd);
  p.part_pre = static_cast<float *>(workspace);
  p.part_post = b ? p.part_pre + static_cast<size_t>(p.units) * static_cast<size_t>(p.ld_part) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch(pl->bwd.fn, dim3(static_cast<unsigned>(p.units)), dim3(pl->bwd.threads), pl->bwd.smem, &p, s) != cudaSuccess) return GE_ERR_CUDA;
  const bool gates = dgate && p.units_per_group;
  if (!dw_pre && !dw_post && !gates) return GE_OK;
  SumParams q;
  std::memset(static_cast<void *>(&q), 0, sizeof(q));
  q.part_pre = p.part_pre;
  q.part_post = p.part_post;
  q.ld_part = p.ld_part;
  q.gate = gate;
  q.w_post = w_post;
  q.dgate = dgate;
  q.dw_post = dw_post;
  q.dw_pre = dw_pre;
  q.alpha = p.alpha;
  q.D = p.D;
  q.wt = p.wt;
  q.units = p.units;
  q.units_per_group = p.units_per_group;
  const int groups = gates ? p.units / p.units_per_group : 0;
  const cudaError_t e = launch(reinterpret_cast<const void *>(norm_sum_kernel),
                               dim3(static_cast<unsigned>(ceil_div(p.D, kSumCols)), static_cast<unsigned>(1 + groups)),
                               dim3(kSumQuads * kSumLanes), 0, &q, s);
  return e == cudaSuccess ? GE_OK : GE_ERR_CUDA;
}

}  // extern "C"
