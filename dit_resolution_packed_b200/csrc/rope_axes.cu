// rope_axes.cu -- host side of pa_rope_axes, and the table of angles for pa_qkv_rope_axes_fwd
// (include/packattn_block.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "host.h"
#include "packattn_block.h"
#include "rope_axes_sm100.cuh"

namespace {

// Frequency and axis of every pair of a head.
pa::RopePairs pairs_of(const pa_rope_axes_desc* r) {
  pa::RopePairs out;
  std::memset(&out, 0, sizeof(out));
  int p = 0;
  for (int a = 0; a < r->axes; ++a)
    for (int i = 0; i < r->dims[a] / 2; ++i, ++p) {
      out.axis[p] = static_cast<int8_t>(a);
      out.turns[p] = std::pow(r->theta[a], -2.0 * i / r->dims[a]) / 6.283185307179586476925286766559;
    }
  out.turned = p;
  for (; p < 64; ++p) out.axis[p] = -1;
  return out;
}

}  // namespace

namespace pa {
namespace host {

int check_rope_axes(const pa_rope_axes_desc* r, int32_t head_dim) {
  if (!r) return PA_ERR_NULL;
  if (r->axes < 1 || r->axes > 4 || (r->interleaved != 0 && r->interleaved != 1)) return PA_ERR_SHAPE;
  int sum = 0;
  for (int a = 0; a < r->axes; ++a) {
    if (r->dims[a] < 2 || r->dims[a] > head_dim || r->dims[a] % 2 != 0) return PA_ERR_SHAPE;
    if (!std::isfinite(r->theta[a]) || r->theta[a] <= 0.0) return PA_ERR_SCALE;
    sum += r->dims[a];
  }
  return sum <= head_dim ? PA_OK : PA_ERR_SHAPE;
}

int rope_turned(const pa_rope_axes_desc* rope) {
  int pairs = 0;
  for (int a = 0; a < rope->axes; ++a) pairs += rope->dims[a] / 2;
  return pairs;
}

int launch_rope_table(const float* pos, int32_t total, int32_t head_dim, const pa_rope_axes_desc* rope, void* table,
                      cudaStream_t stream) {
  pa::RopeTableParams p;
  std::memset(&p, 0, sizeof(p));
  p.pos = pos;
  p.table = static_cast<float2*>(table);
  p.total = total;
  p.half = head_dim / 2;
  p.axes = rope->axes;
  p.pairs = pairs_of(rope);
  const int64_t n = static_cast<int64_t>(total) * p.half;
  pa::rope_axes_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(p);
  return launch_status();
}

}  // namespace host
}  // namespace pa

extern "C" {

int pa_rope_axes(const void* q, const void* k, const float* pos, int32_t total_tokens, int32_t heads, int32_t head_dim,
                 const pa_rope_axes_desc* rope, int32_t inverse, void* q_out, void* k_out, void* stream) {
  if (head_dim != 64 && head_dim != 128) return PA_ERR_HEAD_DIM;
  // a block divides its units (32 bytes each) by those of a token in fp32: exact below 2^22
  if (heads < 1 || total_tokens < 0 || static_cast<int64_t>(heads) * head_dim >= (int64_t(1) << 19)) return PA_ERR_SHAPE;
  if (inverse != 0 && inverse != 1) return PA_ERR_SHAPE;
  int rc = pa::host::check_rope_axes(rope, head_dim);
  if (rc != PA_OK || total_tokens == 0) return rc;
  if (!q || !q_out || !pos || (k == nullptr) != (k_out == nullptr)) return PA_ERR_NULL;
  for (const void* ptr : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (!pa::host::aligned(ptr, 16)) return PA_ERR_ALIGN;
  if (!pa::host::aligned(pos, 4)) return PA_ERR_ALIGN;
  int dev = -1;
  if ((rc = pa::host::common_device({q, k, pos, q_out, k_out}, &dev)) != PA_OK) return rc;
  pa::host::Call call(dev, stream);
  if (call.rc != PA_OK) return call.rc;
  pa::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.in[0] = q;
  p.in[1] = k;
  p.out[0] = q_out;
  p.out[1] = k_out;
  p.pos = pos;
  p.total = total_tokens;
  p.heads = heads;
  p.head_dim = head_dim;
  p.axes = rope->axes;
  p.tensors = k ? 2 : 1;
  p.sign = inverse ? -1.f : 1.f;
  p.pairs = pairs_of(rope);
  const int per_token = heads * (head_dim / 16) * p.tensors;
  p.inv_per_token = 1.f / static_cast<float>(per_token);
  // tokens of a block: about 3 units a thread (measured on 6416 x 24 x 128 and 65536 x 8 x 64: 3 33.6 and 52.0 us,
  // 2 36.8 and 54.3, 4 33.2 and 57.0, 6 35.1 and 63.6, 8 43.3 and 83.8), but enough blocks to fill the GPU
  const int64_t fill = (static_cast<int64_t>(total_tokens) + 4 * call.sms - 1) / (4 * call.sms);
  p.tokens = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>({pa::kRopeAhead * pa::kRopeThreads / per_token, fill, pa::kRopeMaxTokens})));
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(total_tokens) + p.tokens - 1) / p.tokens);
  const bool part = p.pairs.turned < head_dim / 2;
  void (*kernel)(pa::RopeParams) =
      rope->interleaved ? (part ? pa::rope_axes_kernel<true, true> : pa::rope_axes_kernel<true, false>)
                        : (part ? pa::rope_axes_kernel<false, true> : pa::rope_axes_kernel<false, false>);
  kernel<<<grid, pa::kRopeThreads, 0, call.stream>>>(p);
  return pa::host::launch_status();
}

int64_t pa_rope_axes_workspace_bytes(int32_t total_tokens, int32_t head_dim) {
  if (total_tokens < 0 || (head_dim != 64 && head_dim != 128)) return -1;
  return static_cast<int64_t>(total_tokens) * (head_dim / 2) * static_cast<int64_t>(sizeof(float2));
}

}  // extern "C"
