// block_norm_sm100.cuh -- the join between two blocks of a packed stream, and its gradients:
//     u = N_post(y) w_post,   r = residual_scale x + gate[s] u,   z = N_pre(r) w_pre (1 + scale[s]) + shift[s].
//
// A row (token) belongs to a group of W = ceil(C / 256) warps, each thread to 8 neighbouring channels, so a
// row stays in registers between its loads and its stores and the per-channel factors of the current segment
// (gate w_post, (1 + scale) w_pre, shift) are loaded once per segment and kept there too.  The bound is
// memory: every tensor is read once and written once, and each group loads its next row before it works on
// the current one.
//
// Statistics: a warp takes its own mean, then the squares around that mean; the warps' (count, mean, M2) are
// merged with the usual pairwise update, so a row whose mean is far above its deviation loses nothing to
// cancellation and the block needs one exchange through shared memory, not two.
//
// The gradients' column sums (dgate, dscale, dshift) are kept in registers over a chunk of rows and written as
// one fp32 partial per (chunk, segment) to slot chunk + segment: along the stream both only grow and one of
// them does, so no two meet in a slot.  A second kernel adds the slots of a segment in order, a third one
// forms dw_post and dw_pre from the per-segment sums (sum_t dr' gate yhat = sum_s gate[s] sum_{t in s} dr' yhat).
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace pa {

constexpr int kNormMaxHidden = 8192;

struct NormParams {
  const int32_t* cu;  // nullptr: no per-segment factors
  int32_t total, batch, hidden;
  int32_t rows_per_chunk, chunks;
  int32_t warps;   // W of a group
  int32_t post, pre;  // 0 none, 1 layer, 2 rms
  int32_t param_f32;
  float res, eps;
  const void* gate;
  const void* scale;
  const void* shift;
  int64_t gate_stride, scale_stride, shift_stride;
  const void* w_post;
  const void* w_pre;
  const void* x;   // forward: x; backward: r
  const void* y;
  const void* dr;
  const void* dz;
  void* r;         // forward: r; backward: dx
  void* z;         // forward: z; backward: dy
  float* part;     // backward: [chunks + batch][3][C] partial sums (A, B, S), nullptr: no sums wanted
  int32_t* status;
  int32_t err_cu;
};

// Eight channels as they lie in memory, held between their load and their use.
template <bool kF32>
struct Raw8 {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void* p, size_t at) {
    if (kF32) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
      lo = s[0];
      hi = s[1];
    } else {
      lo = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if (kF32) {
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      bf16x8_to_f32(lo, v);
    }
  }
};

// Rounds v to the residual's type in place and stores it.
template <bool kF32>
__device__ __forceinline__ void store8(void* p, size_t at, float (&v)[8]) {
  if (kF32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    const uint4 b = f32_to_bf16x8(v);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = b;
    bf16x8_to_f32(b, v);
  }
}

__device__ __forceinline__ void load_param8(const void* p, size_t at, int f32, float (&v)[8]) {
  if (f32) {
    Raw8<true> a;
    a.load(p, at);
    a.get(v);
  } else {
    Raw8<false> a;
    a.load(p, at);
    a.get(v);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// The exchange of a group's warps: N values per warp through shared memory, double-buffered so that one
// barrier per exchange is enough (a buffer is rewritten two exchanges later, behind the barrier between).
struct GroupLink {
  float (*buf)[32][4];  // [2][warp of the block][4]
  int warps, warp0, warp, group;  // warps of the group, its first warp in the block, own index, group index
  int flip;

  template <int N>
  __device__ __forceinline__ const float (*put(const float (&v)[N], int lane))[4] {
    flip ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[flip][warp0 + warp][i] = v[i];
    }
    named_bar_sync(1 + group, warps * 32);
    return buf[flip] + warp0;
  }
  // Sums of N values over the group (each already summed over its warp), the same order in every thread.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N], int lane) {
    if (warps == 1) return;
    const float(*all)[4] = put<N>(v, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < warps; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += all[w][i];
    }
  }
};

// Mean and M2 (layer) or 0 and the sum of squares (rms) of a warp's channels; `count` of them, >= 8.
__device__ __forceinline__ void warp_moments(const float (&v)[8], bool valid, int kind, float inv_count, float& mean,
                                             float& m2) {
  mean = 0.f;
  if (kind == 1) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
    mean = warp_sum(valid ? s : 0.f) * inv_count;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) q += (v[i] - mean) * (v[i] - mean);
  m2 = warp_sum(valid ? q : 0.f);
}

// Merges the moments of the group's warps: warps 0 .. W-2 hold 256 channels each, the last one the rest.
__device__ __forceinline__ void merge_moments(const float (*all)[4], int at, int warps, int hidden, int kind, float eps,
                                              float& mean, float& rstd) {
  const float inv_c = 1.f / static_cast<float>(hidden);
  float mu = 0.f, m2 = 0.f;
  if (kind == 1) {
    for (int w = 0; w < warps; ++w) mu += all[w][at] * static_cast<float>(min(256, hidden - 256 * w));
    mu *= inv_c;
  }
  for (int w = 0; w < warps; ++w) {
    const float d = all[w][at] - mu;
    m2 += all[w][at + 1] + (kind == 1 ? d * d * static_cast<float>(min(256, hidden - 256 * w)) : 0.f);
  }
  mean = mu;
  rstd = 1.f / sqrtf(m2 * inv_c + eps);
}

// The segment of a token, by a 32-way search of the warp: the last s in [0, batch) with cu[s] <= t (0 if none).
// An empty segment's start equals its successor's, so the last such s is the token's own.
__device__ __forceinline__ int32_t segment_of(const int32_t* cu, int32_t batch, int32_t t, int lane) {
  int32_t lo = 0, n = batch;  // candidates lo .. lo + n - 1
  while (n > 1) {
    const int32_t step = (n + 31) >> 5;
    const int32_t i = lo + lane * step;
    const bool le = lane * step < n && (lane == 0 || cu[i] <= t);
    const int last = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, le)));
    const int32_t off = last * step;
    lo += off;
    n = min(step, n - off);
  }
  return lo;
}

// Records a bad cu_seqlens (one block of the grid does this).
__device__ __forceinline__ void check_cu(const int32_t* cu, int32_t batch, int32_t total, int32_t* status,
                                         int32_t err) {
  if (threadIdx.x == 0 && (cu[0] != 0 || cu[batch] != total)) atomicCAS(status, 0, err);
  for (int32_t i = threadIdx.x; i < batch; i += blockDim.x)
    if (cu[i + 1] < cu[i]) atomicCAS(status, 0, err);
}

// Position of a thread in its block's groups of rows.
struct NormLane {
  int lane, group, groups;
  int32_t chunk;
  int col;
  bool valid;
  float inv_warp;  // 1 / channels of this warp
  __device__ __forceinline__ NormLane(const NormParams& p, GroupLink& link, float (*buf)[32][4]) {
    lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    groups = (blockDim.x >> 5) / p.warps;
    group = w / p.warps;
    link.buf = buf;
    link.warps = p.warps;
    link.group = group;
    link.warp0 = group * p.warps;
    link.warp = w - link.warp0;
    link.flip = 0;
    chunk = blockIdx.x * groups + group;
    col = (link.warp * 32 + lane) * 8;
    valid = col < p.hidden;
    inv_warp = 1.f / static_cast<float>(min(256, p.hidden - 256 * link.warp));
  }
};

template <bool kF32, int kThreads>
__global__ void __launch_bounds__(kThreads) block_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float buf[2][32][4];
  GroupLink link;
  const NormLane me(p, link, buf);
  if (blockIdx.x == 0 && p.cu != nullptr) check_cu(p.cu, p.batch, p.total, p.status, p.err_cu);
  if (me.chunk >= p.chunks) return;  // whole groups leave
  const int64_t row0 = static_cast<int64_t>(me.chunk) * p.rows_per_chunk;
  const int64_t row1 = min(row0 + p.rows_per_chunk, static_cast<int64_t>(p.total));
  const bool join = p.y != nullptr;

  Raw8<kF32> xr;
  Raw8<false> yr;
  const size_t at0 = static_cast<size_t>(row0) * p.hidden + me.col;
  if (me.valid) {
    xr.load(p.x, at0);
    if (join) yr.load(p.y, at0);
  }
  float wpost[8], wpre[8], g[8], a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wpost[i] = wpre[i] = g[i] = a[i] = 1.f;
    b[i] = 0.f;
  }
  if (me.valid) {
    if (p.w_post != nullptr) load_param8(p.w_post, me.col, p.param_f32, wpost);
    if (p.w_pre != nullptr) load_param8(p.w_pre, me.col, p.param_f32, wpre);
  }
  int32_t seg = p.cu != nullptr ? segment_of(p.cu, p.batch, static_cast<int32_t>(row0), me.lane) : 0;
  int64_t seg_end = p.total;
  bool fresh = true;
  for (int64_t row = row0; row < row1; ++row) {
    if (p.cu != nullptr) {
      if (!fresh && row >= seg_end) {
        while (seg + 1 < p.batch && row >= p.cu[seg + 1]) ++seg;
        fresh = true;
      }
      if (fresh) seg_end = seg + 1 < p.batch ? p.cu[seg + 1] : p.total;
    }
    if (fresh) {
      fresh = false;
      if (me.valid) {
        if (p.gate != nullptr) load_param8(p.gate, seg * p.gate_stride + me.col, p.param_f32, g);
        if (p.scale != nullptr) load_param8(p.scale, seg * p.scale_stride + me.col, p.param_f32, a);
        if (p.shift != nullptr) load_param8(p.shift, seg * p.shift_stride + me.col, p.param_f32, b);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] *= wpost[i];
        a[i] = (p.scale != nullptr ? 1.f + a[i] : 1.f) * wpre[i];
      }
      if (p.gate == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = wpost[i];
      }
    }
    float x[8], y[8];
    xr.get(x);
    yr.get(y);
    const size_t at = static_cast<size_t>(row) * p.hidden + me.col;
    if (row + 1 < row1 && me.valid) {
      xr.load(p.x, at + p.hidden);
      if (join) yr.load(p.y, at + p.hidden);
    }
    float mv[2];
    if (join) {
      if (p.post != 0) {
        float mean, rstd;
        warp_moments(y, me.valid, p.post, me.inv_warp, mv[0], mv[1]);
        if (link.warps == 1) {
          mean = mv[0];
          rstd = 1.f / sqrtf(mv[1] / static_cast<float>(p.hidden) + p.eps);
        } else {
          merge_moments(link.put<2>(mv, me.lane), 0, link.warps, p.hidden, p.post, p.eps, mean, rstd);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (y[i] - mean) * rstd;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(p.res, x[i], g[i] * y[i]);
      if (me.valid) store8<kF32>(p.r, at, x);
    }
    if (p.pre != 0) {
      float mean, rstd;
      warp_moments(x, me.valid, p.pre, me.inv_warp, mv[0], mv[1]);
      if (link.warps == 1) {
        mean = mv[0];
        rstd = 1.f / sqrtf(mv[1] / static_cast<float>(p.hidden) + p.eps);
      } else {
        merge_moments(link.put<2>(mv, me.lane), 0, link.warps, p.hidden, p.pre, p.eps, mean, rstd);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf((x[i] - mean) * rstd, a[i], b[i]);
      if (me.valid)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.z) + at) = f32_to_bf16x8(x);
    }
  }
}

// v = N's gradient of an incoming g: rstd (g - [mean g] - hat mean(g hat)), the means over the row's channels.
__device__ __forceinline__ void norm_back(float (&g)[8], const float (&hat)[8], bool valid, int kind, float rstd,
                                          float inv_c, GroupLink& link, int lane) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[0] += g[i];
    s[1] += g[i] * hat[i];
  }
  s[0] = kind == 1 ? warp_sum(valid ? s[0] : 0.f) : 0.f;
  s[1] = warp_sum(valid ? s[1] : 0.f);
  link.sum<2>(s, lane);
  const float c0 = s[0] * inv_c, c1 = s[1] * inv_c;
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = rstd * (g[i] - c0 - hat[i] * c1);
}

template <bool kF32, int kThreads>
__global__ void __launch_bounds__(kThreads) block_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float buf[2][32][4];
  GroupLink link;
  const NormLane me(p, link, buf);
  if (blockIdx.x == 0 && p.cu != nullptr) check_cu(p.cu, p.batch, p.total, p.status, p.err_cu);
  if (me.chunk >= p.chunks) return;
  const int64_t row0 = static_cast<int64_t>(me.chunk) * p.rows_per_chunk;
  const int64_t row1 = min(row0 + p.rows_per_chunk, static_cast<int64_t>(p.total));
  const bool join = p.y != nullptr, front = p.dz != nullptr, given = p.dr != nullptr;
  const float inv_c = 1.f / static_cast<float>(p.hidden);

  Raw8<kF32> rr, drr;
  Raw8<false> yr, dzr;
  const size_t at0 = static_cast<size_t>(row0) * p.hidden + me.col;
  if (me.valid) {
    if (front) {
      rr.load(p.x, at0);
      dzr.load(p.dz, at0);
    }
    if (given) drr.load(p.dr, at0);
    if (join) yr.load(p.y, at0);
  }
  float sa[8], sb[8], ss[8], g[8], a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sa[i] = sb[i] = ss[i] = 0.f;
    g[i] = a[i] = 1.f;
  }
  int32_t seg = p.cu != nullptr ? segment_of(p.cu, p.batch, static_cast<int32_t>(row0), me.lane) : 0;
  int64_t seg_end = p.total;
  bool fresh = true;
  auto flush = [&](int32_t s) {
    if (p.part == nullptr || !me.valid) return;
    float* dst = p.part + (static_cast<size_t>(me.chunk) + s) * 3 * p.hidden + me.col;
    if (join) store8<true>(dst, 0, sa);
    if (front) {
      store8<true>(dst, p.hidden, sb);
      store8<true>(dst, 2 * static_cast<size_t>(p.hidden), ss);
    }
  };
  for (int64_t row = row0; row < row1; ++row) {
    if (p.cu != nullptr) {
      if (!fresh && row >= seg_end) {
        flush(seg);
        while (seg + 1 < p.batch && row >= p.cu[seg + 1]) ++seg;
        fresh = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) sa[i] = sb[i] = ss[i] = 0.f;
      }
      if (fresh) seg_end = seg + 1 < p.batch ? p.cu[seg + 1] : p.total;
    }
    if (fresh) {
      fresh = false;
      if (me.valid) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = a[i] = 1.f;
        if (p.gate != nullptr) load_param8(p.gate, seg * p.gate_stride + me.col, p.param_f32, g);
        if (p.scale != nullptr) {
          load_param8(p.scale, seg * p.scale_stride + me.col, p.param_f32, a);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] += 1.f;
        }
        if (p.w_post != nullptr) {
          load_param8(p.w_post, me.col, p.param_f32, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= w[i];
        }
        if (p.w_pre != nullptr) {
          load_param8(p.w_pre, me.col, p.param_f32, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= w[i];
        }
      }
    }
    float r[8], y[8], dr[8], dz[8];
    rr.get(r);
    yr.get(y);
    drr.get(dr);
    dzr.get(dz);
    const size_t at = static_cast<size_t>(row) * p.hidden + me.col;
    if (row + 1 < row1 && me.valid) {
      const size_t next = at + p.hidden;
      if (front) {
        rr.load(p.x, next);
        dzr.load(p.dz, next);
      }
      if (given) drr.load(p.dr, next);
      if (join) yr.load(p.y, next);
    }
    // the statistics of r and of y in one exchange
    float mv[4] = {0.f, 0.f, 0.f, 0.f};
    float rstd_r = 1.f, rstd_y = 1.f, mean_r = 0.f, mean_y = 0.f;
    if (front) warp_moments(r, me.valid, p.pre, me.inv_warp, mv[0], mv[1]);
    if (join && p.post != 0) warp_moments(y, me.valid, p.post, me.inv_warp, mv[2], mv[3]);
    if (link.warps == 1) {
      mean_r = mv[0];
      mean_y = mv[2];
      rstd_r = 1.f / sqrtf(mv[1] * inv_c + p.eps);
      rstd_y = 1.f / sqrtf(mv[3] * inv_c + p.eps);
    } else if (front || p.post != 0) {
      const float(*all)[4] = link.put<4>(mv, me.lane);
      if (front) merge_moments(all, 0, link.warps, p.hidden, p.pre, p.eps, mean_r, rstd_r);
      if (join && p.post != 0) merge_moments(all, 2, link.warps, p.hidden, p.post, p.eps, mean_y, rstd_y);
    }
    if (!given) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dr[i] = 0.f;
    }
    if (front) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = (r[i] - mean_r) * rstd_r;
        sb[i] += dz[i] * r[i];
        ss[i] += dz[i];
        t[i] = dz[i] * a[i];
      }
      norm_back(t, r, me.valid, p.pre, rstd_r, inv_c, link, me.lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) dr[i] += t[i];
    }
    {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = p.res * dr[i];
      if (me.valid) store8<kF32>(p.r, at, t);
    }
    if (join) {
      if (p.post != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (y[i] - mean_y) * rstd_y;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sa[i] += dr[i] * y[i];
        dr[i] *= g[i];
      }
      if (p.post != 0) norm_back(dr, y, me.valid, p.post, rstd_y, inv_c, link, me.lane);
      if (me.valid)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.z) + at) = f32_to_bf16x8(dr);
    }
  }
  flush(seg);
}

struct NormSumParams {
  const int32_t* cu;  // nullptr: one segment over all tokens
  int32_t total, batch, hidden, rows_per_chunk, chunks, param_f32;
  const float* part;
  float* sums;  // [2][batch][C]: A and B of every segment, nullptr: not needed
  const void* w_post;
  const void* w_pre;
  float* dgate;   // [batch][C], each may be nullptr
  float* dscale;
  float* dshift;
};

// Per segment: the sum of its slots, in order.  One block per (128 channels, segment); its 8 warps take the
// slots 8 apart, then the warps' sums are added in order.
__global__ void __launch_bounds__(256) block_norm_sum_kernel(const __grid_constant__ NormSumParams p) {
  __shared__ float4 acc[3][8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int32_t s = blockIdx.x;
  const int col = blockIdx.y * 128 + lane * 4;
  const bool valid = col < p.hidden;
  const int32_t beg = p.cu != nullptr ? p.cu[s] : 0, end = p.cu != nullptr ? p.cu[s + 1] : p.total;
  int32_t c0 = 0, c1 = 0;  // chunks [c0, c1) of this segment (clamped: cu_seqlens may be bad)
  if (beg >= 0 && end > beg && end <= p.total) {
    c0 = beg / p.rows_per_chunk;
    c1 = min((end - 1) / p.rows_per_chunk + 1, p.chunks);
  }
  const bool use_a = p.dgate != nullptr || (p.sums != nullptr && p.w_post != nullptr);
  const bool use_b = p.dscale != nullptr || (p.sums != nullptr && p.w_pre != nullptr);
  const bool use[3] = {use_a, use_b, p.dshift != nullptr};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (use[k] && valid) {
      for (int32_t c = c0 + w; c < c1; c += 8) {
        const float4 v =
            *reinterpret_cast<const float4*>(p.part + ((static_cast<size_t>(c) + s) * 3 + k) * p.hidden + col);
        t.x += v.x;
        t.y += v.y;
        t.z += v.z;
        t.w += v.w;
      }
    }
    acc[k][w][lane] = t;
  }
  __syncthreads();
  if (w >= 3 || !valid) return;
  const int k = w;
  if (!use[k]) return;
  float4 t = acc[k][0][lane];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    t.x += acc[k][i][lane].x;
    t.y += acc[k][i][lane].y;
    t.z += acc[k][i][lane].z;
    t.w += acc[k][i][lane].w;
  }
  const size_t at = static_cast<size_t>(s) * p.hidden + col;
  if (k < 2 && p.sums != nullptr)
    *reinterpret_cast<float4*>(p.sums + static_cast<size_t>(k) * p.batch * p.hidden + at) = t;
  float* out = k == 0 ? p.dgate : k == 1 ? p.dscale : p.dshift;
  if (out == nullptr) return;
  const void* weight = k == 0 ? p.w_post : k == 1 ? p.w_pre : nullptr;
  float f[4] = {t.x, t.y, t.z, t.w};
  if (weight != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] *= p.param_f32 ? static_cast<const float*>(weight)[col + i]
                          : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(weight)[col + i]) << 16);
  }
  *reinterpret_cast<float4*>(out + at) = make_float4(f[0], f[1], f[2], f[3]);
}

struct NormWeightParams {
  int32_t batch, hidden, param_f32;
  const float* sums;  // [2][batch][C]
  const void* gate;
  const void* scale;
  int64_t gate_stride, scale_stride;
  float* dw_post;
  float* dw_pre;
};

// dw_post = sum_s gate[s] A[s], dw_pre = sum_s (1 + scale[s]) B[s]: one block per 32 channels and weight, its
// 8 warps taking the segments 8 apart.
__global__ void __launch_bounds__(256) block_norm_weight_kernel(const __grid_constant__ NormWeightParams p) {
  __shared__ float acc[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int k = blockIdx.y;
  float* out = k == 0 ? p.dw_post : p.dw_pre;
  if (out == nullptr) return;
  const void* f = k == 0 ? p.gate : p.scale;
  const int64_t stride = k == 0 ? p.gate_stride : p.scale_stride;
  float t = 0.f;
  if (col < p.hidden) {
    const float* src = p.sums + static_cast<size_t>(k) * p.batch * p.hidden + col;
#pragma unroll 4
    for (int32_t s = w; s < p.batch; s += 8) {
      float m = k == 0 ? 1.f : 0.f;
      if (f != nullptr)
        m = p.param_f32
                ? static_cast<const float*>(f)[s * stride + col]
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(f)[s * stride + col]) << 16);
      t += src[static_cast<size_t>(s) * p.hidden] * (k == 0 ? m : 1.f + m);
    }
  }
  acc[w][lane] = t;
  __syncthreads();
  if (w != 0 || col >= p.hidden) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += acc[i][lane];
  out[col] = t;
}

}  // namespace pa
