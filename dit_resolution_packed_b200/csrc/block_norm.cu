// block_norm.cu -- host side of pa_block_norm_fwd and pa_block_norm_bwd (include/packattn_block.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "block_norm_sm100.cuh"
#include "host.h"
#include "packattn_block.h"

namespace {

using pa::host::aligned;

constexpr int kSms = 148;  // the chunking rules below must give one answer for the workspace and the launch

struct Split {
  int32_t warps, groups, rows, chunks;
  int threads() const { return warps * groups * 32; }
};

// A group of warps per row, as many groups as fit 8 warps, and chunks of rows.
Split split_rows(int32_t total, int32_t hidden, int max_rows) {
  Split s;
  s.warps = (hidden + 255) / 256;
  s.groups = std::max(1, 8 / s.warps);
  const int64_t at_once = std::max<int64_t>(1, static_cast<int64_t>(kSms) * 16 / s.warps);
  const int64_t want = (static_cast<int64_t>(total) + 2 * at_once - 1) / (2 * at_once);
  s.rows = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(want, 1), max_rows));
  s.chunks = static_cast<int32_t>((static_cast<int64_t>(total) + s.rows - 1) / s.rows);
  return s;
}
constexpr int kFwdRows = 32;
constexpr int kBwdRows = 64;

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

pa::NormParams params_of(const pa_block_norm_desc* d, const Split& s) {
  pa::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.cu = d->gate || d->scale || d->shift ? d->cu_seqlens : nullptr;
  p.total = d->total_tokens;
  p.batch = p.cu ? d->batch : 1;
  p.hidden = d->hidden;
  p.rows_per_chunk = s.rows;
  p.chunks = s.chunks;
  p.warps = s.warps;
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
  return p;
}

int64_t part_floats(int32_t batch, int32_t hidden, const Split& s) {
  return (static_cast<int64_t>(s.chunks) + std::max(batch, 1)) * 3 * hidden;
}
int64_t sum_floats(int32_t batch, int32_t hidden) { return 2 * static_cast<int64_t>(std::max(batch, 1)) * hidden; }

template <class F>
void by_type(int f32, int threads, F&& launch) {
  // blocks of more than 256 threads hold one row of 2056 channels or more
  if (f32) {
    if (threads <= 256) launch(std::true_type{}, std::integral_constant<int, 256>{});
    else if (threads <= 512) launch(std::true_type{}, std::integral_constant<int, 512>{});
    else launch(std::true_type{}, std::integral_constant<int, 1024>{});
  } else {
    if (threads <= 256) launch(std::false_type{}, std::integral_constant<int, 256>{});
    else if (threads <= 512) launch(std::false_type{}, std::integral_constant<int, 512>{});
    else launch(std::false_type{}, std::integral_constant<int, 1024>{});
  }
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
  const Split s = split_rows(d->total_tokens, d->hidden, kFwdRows);
  pa::NormParams p = params_of(d, s);
  p.x = x;
  p.y = y;
  p.r = r;
  p.z = z;
  p.status = call.status;
  const unsigned grid = static_cast<unsigned>((s.chunks + s.groups - 1) / s.groups);
  by_type(d->residual_fp32, s.threads(), [&](auto f32, auto threads) {
    pa::block_norm_fwd_kernel<f32.value, threads.value><<<grid, s.threads(), 0, call.stream>>>(p);
  });
  return pa::host::launch_status();
}

int64_t pa_block_norm_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t hidden) {
  if (batch < 0 || total_tokens < 0 || hidden < 8 || hidden > pa::kNormMaxHidden || hidden % 8 != 0) return -1;
  const Split s = split_rows(total_tokens, hidden, kBwdRows);
  return 4 * (part_floats(batch, hidden, s) + sum_floats(batch, hidden));
}

int pa_block_norm_bwd(const pa_block_norm_desc* d, const void* r, const void* y, const void* dr, const void* dz,
                      void* dx, void* dy, float* dgate, float* dscale, float* dshift, float* dw_post, float* dw_pre,
                      void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_desc(d);
  if (rc != PA_OK) return rc;
  const bool rows = d->total_tokens > 0;  // without tokens only the sums are memory that the call touches
  if (rows && ((d->pre == PA_NORM_NONE) != (dz == nullptr) || (!dz && !dr))) return PA_ERR_MODE;
  if (rows && (y == nullptr) != (dy == nullptr)) return PA_ERR_MODE;
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
  const Split s = split_rows(d->total_tokens, d->hidden, kBwdRows);
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
  pa::NormParams p = params_of(d, s);
  p.x = r;
  p.y = y;
  p.dr = dr;
  p.dz = dz;
  p.r = dx;
  p.z = dy;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.status = call.status;
  if (rows) {
    const unsigned grid = static_cast<unsigned>((s.chunks + s.groups - 1) / s.groups);
    by_type(d->residual_fp32, s.threads(), [&](auto f32, auto threads) {
      pa::block_norm_bwd_kernel<f32.value, threads.value><<<grid, s.threads(), 0, call.stream>>>(p);
    });
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
  sp.param_f32 = p.param_f32;
  sp.part = p.part;
  sp.sums = weights ? p.part + part_floats(d->batch, d->hidden, s) : nullptr;
  sp.w_post = d->w_post;
  sp.w_pre = d->w_pre;
  sp.dgate = dgate;
  sp.dscale = dscale;
  sp.dshift = dshift;
  pa::block_norm_sum_kernel<<<dim3(p.batch, (p.hidden + 127) / 128), 256, 0, call.stream>>>(sp);
  if ((rc = pa::host::launch_status()) != PA_OK || !weights) return rc;
  pa::NormWeightParams wp;
  std::memset(&wp, 0, sizeof(wp));
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
  pa::block_norm_weight_kernel<<<dim3((p.hidden + 31) / 32, 2), 256, 0, call.stream>>>(wp);
  return pa::host::launch_status();
}

}  // extern "C"
