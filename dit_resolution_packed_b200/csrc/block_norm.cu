// block_norm.cu -- host side of pa_block_norm_fwd and pa_block_norm_bwd (include/packattn_block.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "block_norm_sm100.cuh"
#include "host.h"
#include "packattn_block.h"

namespace {

using pa::host::aligned;

// The splitting rules below give one answer for the workspace and the launch, so they use the number of SMs and of
// warps that the kernels run with on a B200, not what a device reports.
constexpr int kSms = 148;
constexpr int kSmemPerSm = 208 * 1024;  // for rows in flight

int32_t div_up(int32_t a, int32_t b) { return static_cast<int32_t>((static_cast<int64_t>(a) + b - 1) / b); }

// The backward's blocks: teams of threads that own the channels 8 (or 16, 32) a thread, runs of rows, and tiles of
// them with row_warps warps a row; as many rows in flight as shared memory holds.  A thread owns more channels only
// where 8 warps of 8 do not cover a row.  `rows`, `chunks` and `teams` (all
// that the workspace depends on) follow from the sizes alone.
struct BwdSplit {
  int32_t vecs, team_warps, teams, per_sm, rows, chunks;
  int32_t row_bytes, ring_offset, stages, tile, row_warps;
  int threads() const { return 32 * teams * team_warps; }
  size_t smem() const { return ring_offset + static_cast<size_t>(stages) * row_bytes; }
};
BwdSplit split_bwd(int32_t total, int32_t hidden) {
  BwdSplit s;
  std::memset(&s, 0, sizeof(s));
  s.vecs = hidden <= 2048 ? 1 : hidden <= 4096 ? 2 : 4;
  s.team_warps = (hidden + 256 * s.vecs - 1) / (256 * s.vecs);
  s.teams = 8 / s.team_warps;
  s.per_sm = s.vecs == 1 ? 16 / (s.teams * s.team_warps) : 1;  // by the kernels' registers
  s.rows = std::max(1, div_up(total, kSms * s.per_sm));
  s.chunks = div_up(total, s.rows);
  return s;
}
void split_bwd_rows(BwdSplit* s, int32_t hidden, int32_t row_bytes) {
  s->row_bytes = row_bytes;
  s->ring_offset = 8 * hidden;
  const int warps = s->teams * s->team_warps;
  s->stages = std::min(pa::kNormMaxBwdStages,
                       std::max(1, (kSmemPerSm / s->per_sm - s->ring_offset) / std::max(1, row_bytes)));
  // as few warps a row as keep three quarters of the block's warps at work on a tile's rows, and never more than the
  // block has: a group's barrier counts all its warps.  Measured by this rule, with one and with as many warps a row as
  // the block has, us: 16384 x 1152 73, 73, 137; 16384 x 2048 110, 112, 210; 8192 x 4096 108, 118, 157; 4096 x 8192
  // 129, 168, 143.
  s->row_warps = 1;
  while (2 * s->row_warps <= warps && 4 * s->row_warps * std::min(warps / s->row_warps, s->stages) < 3 * warps)
    s->row_warps *= 2;
  s->tile = std::max(1, std::min({warps / s->row_warps, s->stages, pa::kNormMaxTile}));
}

int check_desc(const pa_block_norm_desc* d) {
  if (!d) return PA_ERR_NULL;
  if (d->total_tokens < 0 || d->batch < 0 || (d->batch == 0 && d->total_tokens > 0)) return PA_ERR_SHAPE;
  if (d->hidden < 8 || d->hidden > pa::kNormMaxHidden || d->hidden % 8 != 0) return PA_ERR_SHAPE;
  if (!std::isfinite(d->residual_scale) || !std::isfinite(d->eps) || d->eps < 0.f) return PA_ERR_SCALE;
  if (d->post < PA_NORM_NONE || d->post > PA_NORM_RMS || d->pre < PA_NORM_NONE || d->pre > PA_NORM_RMS ||
      (d->residual_fp32 != 0 && d->residual_fp32 != 1) || (d->param_fp32 != 0 && d->param_fp32 != 1))
    return PA_ERR_MODE;
  if (d->pre == PA_NORM_NONE && (d->w_pre || d->scale || d->shift)) return PA_ERR_MODE;
  const int64_t unit = d->param_fp32 ? 4 : 8;
  const void* mods[3] = {d->gate, d->scale, d->shift};
  const int64_t strides[3] = {d->gate_stride, d->scale_stride, d->shift_stride};
  for (int i = 0; i < 3; ++i) {
    if (!mods[i]) continue;
    if (strides[i] < 0 || strides[i] >= (int64_t(1) << 40)) return PA_ERR_SHAPE;
    if (strides[i] % unit != 0 || !aligned(mods[i], 16)) return PA_ERR_ALIGN;
    if (!d->cu_seqlens) return PA_ERR_NULL;
  }
  if (d->cu_seqlens && !aligned(d->cu_seqlens, 4)) return PA_ERR_ALIGN;
  if (!aligned(d->w_post, 16) || !aligned(d->w_pre, 16)) return PA_ERR_ALIGN;
  return PA_OK;
}

pa::NormParams params_of(const pa_block_norm_desc* d, const pa::host::Call& call) {
  pa::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.cu = d->gate || d->scale || d->shift ? d->cu_seqlens : nullptr;
  p.total = d->total_tokens;
  p.batch = p.cu ? d->batch : 1;
  p.hidden = d->hidden;
  p.post = d->post;
  p.pre = d->pre;
  p.param_f32 = d->param_fp32;
  p.res = d->residual_scale;
  p.eps = d->eps;
  p.gate = d->gate;
  p.scale = d->scale;
  p.shift = d->shift;
  p.gate_stride = d->gate_stride;
  p.scale_stride = d->scale_stride;
  p.shift_stride = d->shift_stride;
  p.w_post = d->w_post;
  p.w_pre = d->w_pre;
  p.err_cu = PA_ERR_CU_SEQLENS;
  p.err_timeout = PA_ERR_TIMEOUT;
  p.status = call.status;
  p.wait_limit_ns = call.wait_limit_ns;
  return p;
}

int64_t part_floats(int32_t batch, int32_t hidden, const BwdSplit& s) {
  return (static_cast<int64_t>(s.chunks) + std::max(batch, 1)) * s.teams * 3 * hidden;
}
int64_t sum_floats(int32_t batch, int32_t hidden) { return 2 * static_cast<int64_t>(std::max(batch, 1)) * hidden; }

// The forward's blocks: one per SM, groups of `warps` warps, each with a ring of rows behind the factors.
// Warps a row: what a row costs whatever its width (shuffles, barriers) is paid by each of its warps, against which
// long rows leave too few in shared memory for one warp each.  Measured with 1, 2 and 4 warps, bf16 / fp32 residual, us:
//     16384 x 1536   42.8 / 57.5   45.6 / 58.0    65.5 / 74.8
//     16384 x 2304   61.7 / 84.1   63.3 / 83.5    78.2 / 91.8
//     16384 x 2560   68.6 / 94.2   67.6 / 91.1    79.2 / 99.5
//      8192 x 3584   57.8 / 85.8   53.2 / 78.2    56.9 / 75.8
//      8192 x 4096   71.4 / 93.0   64.5 / 85.6    60.6 / 81.9
//      4096 x 8192    140 / 237     106 / 175     84.4 / 120
struct FwdSplit {
  int32_t warps, groups, rows, blocks, stages, row_bytes, ring_offset;
  int threads() const { return warps * groups * 32; }
  size_t smem() const { return ring_offset + static_cast<size_t>(groups) * stages * row_bytes; }
};
FwdSplit split_fwd(int32_t total, int32_t hidden, int32_t row_bytes) {
  FwdSplit s;
  s.warps = hidden <= 2304 ? 1 : hidden < 4096 ? 2 : 4;
  s.row_bytes = row_bytes;
  s.ring_offset = 12 * hidden;
  const int room = (kSmemPerSm - s.ring_offset) / row_bytes;  // rows
  const int most = pa::kNormFwdThreads / 32 / s.warps;
  s.rows = div_up(total, kSms);
  // groups for two thirds of the rows that fit (with half as many the same time, with one for every row no better), no
  // more than rows, and whole stages of what fits for each: more than one only where `most` or the rows limit the groups
  // (joined rows below about 1050 bf16 or 710 fp32 channels, or a short pack).  With one stage a group asks for its next
  // row when it is done with the current one, and what overlaps the copy is the other groups' work.
  s.groups = std::max(1, std::min({most, room * 2 / 3, s.rows}));
  s.stages = std::max(1, std::min(pa::kNormMaxStages, room / s.groups));
  s.blocks = div_up(total, s.rows);
  return s;
}

// The kernels of a type, and of a split's warps (forward) or vectors (backward).
template <bool kF32>
struct Kernels {
  static constexpr auto fwd1 = pa::block_norm_fwd_kernel<kF32, 1>;
  static constexpr auto fwd2 = pa::block_norm_fwd_kernel<kF32, 2>;
  static constexpr auto fwd4 = pa::block_norm_fwd_kernel<kF32, 4>;
  static constexpr auto bwd1 = pa::block_norm_bwd_kernel<kF32, 1>;
  static constexpr auto bwd2 = pa::block_norm_bwd_kernel<kF32, 2>;
  static constexpr auto bwd4 = pa::block_norm_bwd_kernel<kF32, 4>;
  static void (*fwd(int warps))(pa::NormFwdParams) { return warps == 1 ? fwd1 : warps == 2 ? fwd2 : fwd4; }
  static void (*bwd(int vecs))(pa::NormBwdParams) { return vecs == 1 ? bwd1 : vecs == 2 ? bwd2 : bwd4; }
  static bool allow_smem() {
    for (int w : {1, 2, 4})
      if (cudaFuncSetAttribute(fwd(w), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm) != cudaSuccess)
        return false;
    for (int v : {1, 2, 4})
      if (cudaFuncSetAttribute(bwd(v), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm) != cudaSuccess)
        return false;
    return true;
  }
};
// Shared-memory limits, once per device (the caller holds the library's lock).
int ensure_kernels(int dev) {
  static bool ready[64] = {};
  if (ready[dev]) return PA_OK;
  if (!Kernels<false>::allow_smem() || !Kernels<true>::allow_smem()) return PA_ERR_CUDA;
  ready[dev] = true;
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_block_norm_fwd(const pa_block_norm_desc* d, const void* x, const void* y, void* r, void* z, void* stream) {
  int rc = check_desc(d);
  if (rc != PA_OK) return rc;
  if (d->total_tokens == 0) return PA_OK;
  if ((d->pre == PA_NORM_NONE) != (z == nullptr)) return PA_ERR_MODE;
  if (!y && (r || d->post != PA_NORM_NONE || d->w_post || d->gate || d->residual_scale != 1.f || !z)) return PA_ERR_MODE;
  if (!x || (y && !r)) return PA_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(r, 16) || !aligned(z, 16)) return PA_ERR_ALIGN;
  int dev = -1;
  const bool per_segment = d->gate || d->scale || d->shift;
  if ((rc = pa::host::common_device({x, y, r, z, d->gate, d->scale, d->shift, d->w_post, d->w_pre,
                                     per_segment ? d->cu_seqlens : nullptr},
                                    &dev)) != PA_OK)
    return rc;
  pa::host::Call call(dev, stream);
  if (call.rc != PA_OK) return call.rc;
  if ((rc = ensure_kernels(dev)) != PA_OK) return rc;
  const FwdSplit s = split_fwd(d->total_tokens, d->hidden, d->hidden * ((d->residual_fp32 ? 4 : 2) + (y ? 2 : 0)));
  pa::NormFwdParams f;
  f.n = params_of(d, call);
  f.n.rows_per_chunk = s.rows;
  f.n.chunks = s.blocks;
  f.n.stages = s.stages;
  f.n.row_bytes = s.row_bytes;
  f.n.x = x;
  f.n.y = y;
  f.n.r = r;
  f.n.z = z;
  f.groups = s.groups;
  f.ring_offset = s.ring_offset;
  const auto kernel = d->residual_fp32 ? Kernels<true>::fwd(s.warps) : Kernels<false>::fwd(s.warps);
  kernel<<<s.blocks, s.threads(), s.smem(), call.stream>>>(f);
  return pa::host::launch_status();
}

int64_t pa_block_norm_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t hidden) {
  if (batch < 0 || total_tokens < 0 || hidden < 8 || hidden > pa::kNormMaxHidden || hidden % 8 != 0) return -1;
  const BwdSplit s = split_bwd(total_tokens, hidden);
  return 4 * (part_floats(batch, hidden, s) + sum_floats(batch, hidden));
}

int pa_block_norm_bwd(const pa_block_norm_desc* d, const void* r, const void* y, const void* dr, const void* dz,
                      void* dx, void* dy, float* dgate, float* dscale, float* dshift, float* dw_post, float* dw_pre,
                      void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_desc(d);
  if (rc != PA_OK) return rc;
  const bool rows = d->total_tokens > 0;  // without tokens only the sums are memory that the call touches
  if (rows && ((d->pre == PA_NORM_NONE) != (dz == nullptr) || (!dz && !dr))) return PA_ERR_MODE;
  if (rows && ((y == nullptr) != (dy == nullptr) || (!y && !dz))) return PA_ERR_MODE;
  if (rows && !y && (d->post != PA_NORM_NONE || d->w_post || d->gate || d->residual_scale != 1.f)) return PA_ERR_MODE;
  if ((dgate && !d->gate) || (dscale && !d->scale) || (dshift && !d->shift) || (dw_post && !d->w_post) ||
      (dw_pre && !d->w_pre))
    return PA_ERR_MODE;
  const bool sums = dgate || dscale || dshift || dw_post || dw_pre;
  const bool weights = dw_post || dw_pre;
  if (!rows && !sums) return PA_OK;
  if (rows && ((dz && !r) || !dx)) return PA_ERR_NULL;
  for (const void* ptr : {r, y, dr, dz, static_cast<const void*>(dx), static_cast<const void*>(dy),
                          static_cast<const void*>(dgate), static_cast<const void*>(dscale),
                          static_cast<const void*>(dshift), static_cast<const void*>(dw_post),
                          static_cast<const void*>(dw_pre)})
    if (!aligned(ptr, 16)) return PA_ERR_ALIGN;
  BwdSplit s = split_bwd(d->total_tokens, d->hidden);
  const int32_t wide = d->residual_fp32 ? 4 : 2;
  split_bwd_rows(&s, d->hidden, d->hidden * ((dz ? wide + 2 : 0) + (dr ? wide : 0) + (y ? 2 : 0)));
  if (sums) {
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pa_block_norm_workspace_bytes(d->batch, d->total_tokens, d->hidden))
      return PA_ERR_WORKSPACE;
  }
  int dev = -1;
  const bool per_segment = d->gate || d->scale || d->shift;
  if ((rc = pa::host::common_device({rows ? r : nullptr, rows ? y : nullptr, rows ? dr : nullptr, rows ? dz : nullptr,
                                     rows ? dx : nullptr, rows ? dy : nullptr, dgate, dscale, dshift, dw_post, dw_pre,
                                     sums ? workspace : nullptr, d->gate, d->scale, d->shift, d->w_post, d->w_pre,
                                     per_segment ? d->cu_seqlens : nullptr},
                                    &dev)) != PA_OK)
    return rc;
  pa::host::Call call(dev, stream);
  if (call.rc != PA_OK) return call.rc;
  if ((rc = ensure_kernels(dev)) != PA_OK) return rc;
  pa::NormBwdParams b;
  b.n = params_of(d, call);
  b.tile = s.tile;
  b.row_warps = s.row_warps;
  b.teams = s.teams;
  b.team_warps = s.team_warps;
  b.ring_offset = s.ring_offset;
  pa::NormParams& p = b.n;
  p.rows_per_chunk = s.rows;
  p.chunks = s.chunks;
  p.stages = s.stages;
  p.row_bytes = s.row_bytes;
  p.x = r;
  p.y = y;
  p.dr = dr;
  p.dz = dz;
  p.r = dx;
  p.z = dy;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  if (rows) {
    const auto kernel = d->residual_fp32 ? Kernels<true>::bwd(s.vecs) : Kernels<false>::bwd(s.vecs);
    kernel<<<s.chunks, s.threads(), s.smem(), call.stream>>>(b);
    if ((rc = pa::host::launch_status()) != PA_OK) return rc;
  }
  if (!sums) return PA_OK;
  if (p.batch == 0) {  // no segment: only the weights' gradients have a size
    for (float* w : {dw_post, dw_pre})
      if (w && cudaMemsetAsync(w, 0, 4 * static_cast<size_t>(d->hidden), call.stream) != cudaSuccess)
        return PA_ERR_CUDA;
    return PA_OK;
  }
  pa::NormSumParams sp;
  std::memset(&sp, 0, sizeof(sp));
  sp.cu = p.cu;
  sp.total = p.total;
  sp.batch = p.batch;
  sp.hidden = p.hidden;
  sp.rows_per_chunk = p.rows_per_chunk;
  sp.chunks = p.chunks;
  sp.teams = s.teams;
  sp.param_f32 = p.param_f32;
  sp.part = p.part;
  sp.sums = weights ? p.part + part_floats(d->batch, d->hidden, s) : nullptr;
  sp.w_post = d->w_post;
  sp.w_pre = d->w_pre;
  sp.dgate = dgate;
  sp.dscale = dscale;
  sp.dshift = dshift;
  sp.use = (dgate || dw_post ? 1 : 0) | (dscale || dw_pre ? 2 : 0) | (dshift ? 4 : 0);
  // Some 40 segments fill the GPU; with fewer, every segment's slots are read in parallel.  The whole backward of
  // 65536 x 1152 by one and the other: 3 segments 195 and 196 us, 16 204 and 195, 24 202 and 198, 32 200 and 198, 48 199
  // and 200, 256 198 and 231, 2048 223 and 492.  (A long one among many has blocks of its own: the kernel.)
  if (p.batch > 40) {
    const int32_t by = div_up(p.hidden, 4 * pa::kNormSumThreads);
    sp.long_runs = std::max(1, 32 / s.teams);  // 32 slots, one for each part of a long segment
    sp.long_col_blocks = div_up(p.hidden, 32 * by);
    const int64_t blocks = p.batch + static_cast<int64_t>(div_up(p.chunks, sp.long_runs)) * sp.long_col_blocks;
    rc = pa::host::launch_behind(pa::block_norm_sum_kernel, dim3(static_cast<unsigned>(blocks), by), pa::kNormSumThreads,
                                 0, call.stream, sp);
  } else
    rc = pa::host::launch_behind(pa::block_norm_sum_long_kernel, dim3(p.batch, (p.hidden + 127) / 128),
                                 pa::kNormSumLongThreads, 0, call.stream, sp);
  if (rc != PA_OK || !weights) return rc;
  pa::NormWeightParams wp;
  std::memset(&wp, 0, sizeof(wp));
  wp.cu = p.cu;
  wp.batch = p.batch;
  wp.hidden = p.hidden;
  wp.param_f32 = p.param_f32;
  wp.sums = sp.sums;
  wp.gate = d->gate;
  wp.scale = d->scale;
  wp.gate_stride = d->gate_stride;
  wp.scale_stride = d->scale_stride;
  wp.dw_post = dw_post;
  wp.dw_pre = dw_pre;
  return pa::host::launch_behind(pa::block_norm_weight_kernel, dim3((p.hidden + 31) / 32, 2), 256, 0, call.stream, wp);
}

}  // extern "C"
