// sparse.cu -- host side of pa_block_select and pa_block_sparse_attn_fwd / _bwd (include/packattn_block.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_bwd_sm100.cuh"
#include "attn_sparse_fwd_sm100.cuh"
#include "host.h"
#include "packattn_block.h"
#include "sparse_plan_sm100.cuh"

namespace {

using pa::host::aligned;

constexpr int64_t kAlign = 256;
int64_t up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// The caller's workspace begins at any 16-byte boundary; its parts at the next 256-byte one.
uint8_t* base_of(void* ws) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + kAlign - 1) / kAlign * kAlign);
}

int64_t block_rows(int32_t batch, int32_t total) { return static_cast<int64_t>(total) / 128 + batch; }
int64_t pair_rows(int32_t batch, int32_t total) { return static_cast<int64_t>(total) / 256 + batch; }

// Byte offsets of a plan's parts.  The backward zeroes [0, cleared) before its plan kernels run.
struct Layout {
  int64_t counts, bits, cleared, cls, order, desc, steps, maps, lse2, delta, dq, total;
  int32_t words;
};

Layout layout(int32_t batch, int32_t total, int32_t heads, int32_t head_dim, int32_t max_seqlen, int32_t width,
              bool backward) {
  Layout L;
  const int64_t items = heads * (backward ? block_rows(batch, total) : pair_rows(batch, total));
  const int64_t rows = static_cast<int64_t>(total) * heads;
  L.words = (std::min(max_seqlen, total) + 4095) / 4096;  // 32 blocks of 128 tokens a word
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes);
    return here;
  };
  L.counts = take(16);
  L.bits = take(backward ? 4 * items * L.words : 0);
  L.cleared = at;
  L.cls = take(4 * items);  // (parts are padded to 256 bytes: it is read 16 at a time)
  L.order = take(4 * items);
  L.desc = take(4 * pa::kDescInts * items);
  L.steps = take(backward ? 0 : 8 * items * width);
  L.maps = take(static_cast<int64_t>(batch) * (backward ? 4 : 3) * 128);
  L.lse2 = take(backward ? 4 * rows : 0);
  L.delta = take(backward ? 4 * rows : 0);
  L.dq = take(backward ? 4 * rows * head_dim : 0);
  L.total = at + kAlign;  // for the base's alignment
  return L;
}

bool sizes_ok(int32_t batch, int32_t total, int32_t heads, int32_t head_dim) {
  return heads >= 1 && batch >= 0 && total >= 0 && !(batch == 0 && total > 0) &&
         static_cast<int64_t>(heads) * head_dim < (int64_t(1) << 23) &&
         block_rows(batch, total) * heads < (int64_t(1) << 31) &&
         static_cast<int64_t>(total) * heads * head_dim < (int64_t(1) << 40);
}

// Entries of a list table (sizes_ok holds): few enough that no size formed of them passes 63 bits.
bool table_ok(int32_t batch, int32_t total, int32_t heads, int32_t width) {
  return block_rows(batch, total) * heads <= (int64_t(1) << 40) / std::max(width, 1);
}

int32_t keep_count(int32_t nb, double density, int32_t min_blocks) {
  return std::min(nb, std::max(min_blocks, static_cast<int32_t>(std::ceil(density * static_cast<double>(nb)))));
}

// Shared memory of select_topk_kernel: the group's query means, a chunk of key means, the warps' parts, the scores.
size_t topk_smem(int32_t head_dim, int32_t nb) {
  return 8 * (8 * static_cast<size_t>(head_dim) + 32 * (static_cast<size_t>(head_dim) + 2) + 8 * 8 * 32 +
              8 * static_cast<size_t>(nb));
}

// Shared-memory limits of this file's kernels, once per device (the caller holds the library's lock).
int ensure_kernels(int dev) {
  static bool ready[64] = {};
  if (ready[dev]) return PA_OK;
  auto big = [](const void* f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  const int topk = static_cast<int>(topk_smem(128, pa::kSelectMaxBlocks));
  if (!big(reinterpret_cast<const void*>(pa::attn_sparse_fwd_kernel<64>), pa::FwdCfg<64>::kSmemBytes) ||
      !big(reinterpret_cast<const void*>(pa::attn_sparse_fwd_kernel<128>), pa::FwdCfg<128>::kSmemBytes) ||
      !big(reinterpret_cast<const void*>(pa::attn_bwd_kernel<64, true>), pa::BwdCfg<64>::kSmemBytes) ||
      !big(reinterpret_cast<const void*>(pa::attn_bwd_kernel<128, true>), pa::BwdCfg<128>::kSmemBytes) ||
      !big(reinterpret_cast<const void*>(pa::select_topk_kernel<64>), topk) ||
      !big(reinterpret_cast<const void*>(pa::select_topk_kernel<128>), topk))
    return PA_ERR_CUDA;
  ready[dev] = true;
  return PA_OK;
}

// The plan's parameters but for the maps' bases.
pa::SparsePlanParams plan_params(const Layout& L, uint8_t* ws, const int32_t* cu, const int32_t* idx,
                                 const int32_t* cnt, int32_t batch, int32_t total, int32_t heads, int32_t head_dim,
                                 int32_t max_seqlen, int32_t width, bool backward, int32_t* status) {
  pa::SparsePlanParams p;
  std::memset(&p, 0, sizeof(p));
  p.cu = cu;
  p.idx = idx;
  p.cnt = cnt;
  p.batch = batch;
  p.total = total;
  p.heads = heads;
  p.max_seqlen = max_seqlen;
  p.width = width;
  p.n_maps = backward ? 4 : 3;
  p.rows = block_rows(batch, total);
  p.units = backward ? p.rows : pair_rows(batch, total);
  p.row_bytes = static_cast<uint64_t>(heads) * head_dim * 2;
  p.counts = reinterpret_cast<int32_t*>(ws + L.counts);
  p.cls = reinterpret_cast<int32_t*>(ws + L.cls);
  p.order = reinterpret_cast<int32_t*>(ws + L.order);
  p.desc = reinterpret_cast<int32_t*>(ws + L.desc);
  p.steps = reinterpret_cast<int2*>(ws + L.steps);
  p.bits = reinterpret_cast<uint32_t*>(ws + L.bits);
  p.words = L.words;
  p.maps = ws + L.maps;
  p.status = status;
  p.err_cu = PA_ERR_CU_SEQLENS;
  p.err_max = PA_ERR_MAX_SEQLEN;
  p.err_blocks = PA_ERR_BLOCKS;
  return p;
}

unsigned warps4(int64_t n) { return static_cast<unsigned>((n + 3) / 4); }

}  // namespace

extern "C" {

int64_t pa_block_rows(int32_t batch, int32_t total_tokens) {
  if (batch < 0 || total_tokens < 0) return -1;
  return block_rows(batch, total_tokens);
}

int64_t pa_block_select_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t heads, int32_t head_dim) {
  if ((head_dim != 64 && head_dim != 128) || !sizes_ok(batch, total_tokens, heads, head_dim)) return -1;
  return 2 * 8 * block_rows(batch, total_tokens) * heads * head_dim;
}

int pa_block_select(const void* q, const void* k, const int32_t* cu_seqlens, int32_t batch, int32_t total_tokens,
                    int32_t heads, int32_t head_dim, int32_t max_seqlen, double density, int32_t min_blocks,
                    int32_t width, int32_t* idx, int32_t* cnt, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
  if (!sizes_ok(batch, total_tokens, heads, head_dim) || heads > 65535 || min_blocks < 1 || width < 1 ||
      !table_ok(batch, total_tokens, heads, width))
    return PA_ERR_SHAPE;
  if (!(density >= 0.0 && density <= 1.0)) return PA_ERR_SCALE;
  if (batch == 0) return PA_OK;
  if (!idx || !cnt) return PA_ERR_NULL;
  if (!aligned(idx, 4) || !aligned(cnt, 4)) return PA_ERR_ALIGN;
  const int64_t rows = block_rows(batch, total_tokens);
  int rc, dev = -1;
  if (total_tokens == 0) {  // every row is no block
    if ((rc = pa::host::common_device({idx, cnt}, &dev)) != PA_OK) return rc;
    pa::host::Call call(dev, stream);
    if (call.rc != PA_OK) return call.rc;
    const size_t n = 4 * static_cast<size_t>(rows) * heads;
    return cudaMemsetAsync(cnt, 0, n, call.stream) == cudaSuccess &&
                   cudaMemsetAsync(idx, 0xff, n * width, call.stream) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  }
  if (max_seqlen < 1) return PA_ERR_MAX_SEQLEN;
  const int32_t longest = std::min(max_seqlen, total_tokens);
  const int32_t nb = (longest + 127) / 128;
  if (nb > pa::kSelectMaxBlocks) return PA_ERR_MAX_SEQLEN;
  if (width < keep_count(nb, density, min_blocks)) return PA_ERR_BLOCKS;
  if (!q || !k || !cu_seqlens) return PA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(cu_seqlens, 4)) return PA_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 16) ||
      workspace_bytes < pa_block_select_workspace_bytes(batch, total_tokens, heads, head_dim))
    return PA_ERR_WORKSPACE;
  if ((rc = pa::host::common_device({q, k, cu_seqlens, idx, cnt, workspace}, &dev)) != PA_OK) return rc;
  pa::host::Call call(dev, stream);
  if (call.rc != PA_OK) return call.rc;
  if ((rc = ensure_kernels(dev)) != PA_OK) return rc;
  pa::SelectParams p;
  std::memset(&p, 0, sizeof(p));
  p.x[0] = static_cast<const uint16_t*>(q);
  p.x[1] = static_cast<const uint16_t*>(k);
  p.cu = cu_seqlens;
  p.batch = batch;
  p.total = total_tokens;
  p.heads = heads;
  p.head_dim = head_dim;
  p.max_seqlen = longest;
  p.width = width;
  p.min_blocks = min_blocks;
  p.density = density;
  p.mean = static_cast<double*>(workspace);
  p.rows = rows;
  p.idx = idx;
  p.cnt = cnt;
  p.status = call.status;
  p.err_cu = PA_ERR_CU_SEQLENS;
  p.err_max = PA_ERR_MAX_SEQLEN;
  const int32_t channels = heads * head_dim;
  pa::select_pool_kernel<<<dim3(static_cast<unsigned>(rows), (channels + 255) / 256, 2), pa::kPoolThreads, 0,
                           call.stream>>>(p);
  if ((rc = pa::host::launch_status()) != PA_OK) return rc;
  const dim3 grid(static_cast<unsigned>(total_tokens / 1024 + batch), heads);
  const size_t smem = topk_smem(head_dim, nb);
  return pa::host::launch_behind(head_dim == 128 ? pa::select_topk_kernel<128> : pa::select_topk_kernel<64>, grid, 256, smem,
                                 call.stream, p);
}

int64_t pa_block_sparse_workspace_bytes(int32_t batch, int32_t total_tokens, int32_t heads, int32_t head_dim,
                                        int32_t max_seqlen, int32_t width, int32_t backward) {
  if ((head_dim != 64 && head_dim != 128) || !sizes_ok(batch, total_tokens, heads, head_dim) || width < 0 ||
      max_seqlen < 0 || !table_ok(batch, total_tokens, heads, width))
    return -1;
  return layout(batch, total_tokens, heads, head_dim, max_seqlen, width, backward != 0).total;
}

int pa_block_sparse_attn_fwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int32_t batch,
                             int32_t total_tokens, int32_t heads, int32_t head_dim, int32_t max_seqlen,
                             const int32_t* idx, const int32_t* cnt, int32_t width, float scale, void* out, float* lse,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
  if (!sizes_ok(batch, total_tokens, heads, head_dim) || width < 1 || !table_ok(batch, total_tokens, heads, width))
    return PA_ERR_SHAPE;
  if (!std::isfinite(scale)) return PA_ERR_SCALE;
  if (batch == 0 || total_tokens == 0) return PA_OK;
  if (max_seqlen < 1) return PA_ERR_MAX_SEQLEN;
  if (!q || !k || !v || !cu_seqlens || !idx || !cnt || !out || !lse) return PA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(idx, 4) || !aligned(cnt, 4))
    return PA_ERR_ALIGN;
  const Layout L = layout(batch, total_tokens, heads, head_dim, max_seqlen, width, false);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total) return PA_ERR_WORKSPACE;
  int rc, dev = -1;
  if ((rc = pa::host::common_device({q, k, v, cu_seqlens, idx, cnt, out, lse, workspace}, &dev)) != PA_OK) return rc;
  pa::host::Call call(dev, stream);
  if (call.rc != PA_OK) return call.rc;
  if ((rc = ensure_kernels(dev)) != PA_OK) return rc;
  uint8_t* ws = base_of(workspace);
  pa::SparsePlanParams p = plan_params(L, ws, cu_seqlens, idx, cnt, batch, total_tokens, heads, head_dim, max_seqlen,
                                       width, false, call.status);
  const void* bases[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    if (!pa::host::encode_rows(&p.tmpl[i], bases[i], total_tokens, heads, head_dim) ||
        !pa::host::encode_rows(&p.small[i], bases[i], 1, heads, head_dim))
      return PA_ERR_CUDA;
    p.base[i] = bases[i];
  }
  const int64_t items = p.units * heads;
  // With no more items than CTAs all run at once and their order is of no use: a launch fewer (364 tokens, 2 heads:
  // 17.7 us against 21.0 on the GPU).
  p.sorted = items > call.sms ? 1 : 0;
  pa::sparse_plan_fwd_kernel<<<warps4(items), 128, 0, call.stream>>>(p);
  if ((rc = pa::host::launch_status()) != PA_OK) return rc;
  if (p.sorted && (rc = pa::host::launch_behind(pa::sparse_order_kernel, pa::kSparseClasses, pa::kOrderThreads, 0, call.stream,
                                                p)) != PA_OK)
    return rc;
  pa::SparseFwdParams f;
  std::memset(&f, 0, sizeof(f));
  f.counts = p.counts;
  f.next_item = p.counts + 2;
  f.order = p.sorted ? p.order : nullptr;
  f.desc = p.desc;
  f.steps = p.steps;
  f.maps = p.maps;
  f.out = out;
  f.lse = lse;
  f.status = call.status;
  f.heads = heads;
  f.width = width;
  f.out32 = aligned(out, 32) ? 1 : 0;
  f.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  f.wait_limit_ns = call.wait_limit_ns;
  f.err_timeout = PA_ERR_TIMEOUT;
  return pa::host::launch_behind(head_dim == 128 ? pa::attn_sparse_fwd_kernel<128> : pa::attn_sparse_fwd_kernel<64>,
                                 static_cast<unsigned>(std::min<int64_t>(call.sms, items)), pa::kFwdThreads,
                                 head_dim == 128 ? pa::FwdCfg<128>::kSmemBytes : pa::FwdCfg<64>::kSmemBytes, call.stream,
                                 f);
}

int pa_block_sparse_attn_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse,
                             const void* dout, const int32_t* cu_seqlens, int32_t batch, int32_t total_tokens,
                             int32_t heads, int32_t head_dim, int32_t max_seqlen, const int32_t* idx,
                             const int32_t* cnt, int32_t width, float scale, void* dq, void* dk, void* dv,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
  if (!sizes_ok(batch, total_tokens, heads, head_dim) || width < 1 || !table_ok(batch, total_tokens, heads, width))
    return PA_ERR_SHAPE;
  if (!std::isfinite(scale)) return PA_ERR_SCALE;
  if (batch == 0 || total_tokens == 0) return PA_OK;
  if (max_seqlen < 1) return PA_ERR_MAX_SEQLEN;
  if (!q || !k || !v || !out || !lse || !dout || !cu_seqlens || !idx || !cnt || !dq || !dk || !dv) return PA_ERR_NULL;
  const void* a16[8] = {q, k, v, out, dout, dq, dk, dv};
  for (const void* ptr : a16)
    if (!aligned(ptr, 16)) return PA_ERR_ALIGN;
  if (!aligned(lse, 4) || !aligned(cu_seqlens, 4) || !aligned(idx, 4) || !aligned(cnt, 4)) return PA_ERR_ALIGN;
  const Layout L = layout(batch, total_tokens, heads, head_dim, max_seqlen, width, true);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total) return PA_ERR_WORKSPACE;
  int rc, dev = -1;
  if ((rc = pa::host::common_device({q, k, v, out, lse, dout, cu_seqlens, idx, cnt, dq, dk, dv, workspace}, &dev)) !=
      PA_OK)
    return rc;
  pa::host::Call call(dev, stream);
  if (call.rc != PA_OK) return call.rc;
  if ((rc = ensure_kernels(dev)) != PA_OK) return rc;
  uint8_t* ws = base_of(workspace);
  pa::SparsePlanParams p = plan_params(L, ws, cu_seqlens, idx, cnt, batch, total_tokens, heads, head_dim, max_seqlen,
                                       width, true, call.status);
  const void* bases[4] = {q, k, v, dout};
  for (int i = 0; i < 4; ++i) {
    if (!pa::host::encode_rows(&p.tmpl[i], bases[i], total_tokens, heads, head_dim) ||
        !pa::host::encode_rows(&p.small[i], bases[i], 1, heads, head_dim))
      return PA_ERR_CUDA;
    p.base[i] = bases[i];
  }
  const int64_t items = p.units * heads;
  p.sorted = 1;
  if (cudaMemsetAsync(ws, 0, L.cleared, call.stream) != cudaSuccess) return PA_ERR_CUDA;
  pa::sparse_mark_kernel<<<warps4(items), 128, 0, call.stream>>>(p);
  if ((rc = pa::host::launch_status()) != PA_OK) return rc;
  if ((rc = pa::host::launch_behind(pa::sparse_plan_bwd_kernel, warps4(items), 128, 0, call.stream, p)) != PA_OK ||
      (rc = pa::host::launch_behind(pa::sparse_order_kernel, pa::kSparseClasses, pa::kOrderThreads, 0, call.stream, p)) !=
          PA_OK)
    return rc;

  float* lse2 = reinterpret_cast<float*>(ws + L.lse2);
  float* delta = reinterpret_cast<float*>(ws + L.delta);
  float* dq_acc = reinterpret_cast<float*>(ws + L.dq);
  const int64_t rows = static_cast<int64_t>(total_tokens) * heads;
  const int64_t acc_n4 = rows * (head_dim / 4);
  const int64_t prep_warps = (rows + pa::kPrepRowsPerWarp - 1) / pa::kPrepRowsPerWarp;
  const unsigned prep_blocks = static_cast<unsigned>((prep_warps * 32 + 255) / 256);
  auto prep = head_dim == 128 ? pa::bwd_prep_kernel<128> : pa::bwd_prep_kernel<64>;
  prep<<<prep_blocks, 256, 0, call.stream>>>(static_cast<const uint16_t*>(out), static_cast<const uint16_t*>(dout), lse,
                                            delta, lse2, reinterpret_cast<float4*>(dq_acc), acc_n4, total_tokens,
                                            heads);
  if ((rc = pa::host::launch_status()) != PA_OK) return rc;

  pa::BwdParams b;
  std::memset(&b, 0, sizeof(b));
  b.counts = p.counts;
  b.next_item = p.counts + 2;
  b.order = p.order;
  b.lse2 = lse2;
  b.delta = delta;
  b.dq_acc = dq_acc;
  b.dk = dk;
  b.dv = dv;
  b.status = call.status;
  b.heads = heads;
  b.total = total_tokens;
  b.scale = scale;
  b.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  b.wait_limit_ns = call.wait_limit_ns;
  b.err_timeout = PA_ERR_TIMEOUT;
  b.desc = p.desc;
  b.bits = p.bits;
  b.words = p.words;
  b.out32 = aligned(dk, 32) && aligned(dv, 32) ? 1 : 0;
  b.maps = p.maps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(call.sms, items));
  void (*kernel)(pa::BwdParams) = head_dim == 128 ? pa::attn_bwd_kernel<128, true> : pa::attn_bwd_kernel<64, true>;
  if ((rc = pa::host::launch_behind(kernel, grid, pa::kBwdThreads,
                                    head_dim == 128 ? pa::BwdCfg<128>::kSmemBytes : pa::BwdCfg<64>::kSmemBytes,
                                    call.stream, b)) != PA_OK)
    return rc;

  const unsigned conv = static_cast<unsigned>(((static_cast<int64_t>(total_tokens) + 31) / 32) * heads);
  auto convert = head_dim == 128 ? pa::bwd_dq_convert_kernel<128> : pa::bwd_dq_convert_kernel<64>;
  convert<<<conv, 256, 0, call.stream>>>(reinterpret_cast<const float4*>(dq_acc), static_cast<uint16_t*>(dq),
                                         total_tokens, heads);
  return pa::host::launch_status();
}

}  // extern "C"
