// block_norm_sm100.cuh -- the join between two blocks of a packed stream, and its gradients:
//     u = N_post(y) w_post,   r = residual_scale x + gate[s] u,   z = N_pre(r) w_pre (1 + scale[s]) + shift[s].
//
// The bound is memory: every tensor is read once and written once.  A block takes a run of neighbouring rows (tokens),
// which bulk copies bring into shared memory, so the bytes in flight do not depend on registers: as many rows as fit, some
// of them worked on and the others on their way.
//
// Statistics: a warp sums its channels and their squares around a pivot of its own (the mean of its first sweep of
// 256), which gives its (mean, M2); where several warps share a row, theirs are merged the same way around the first
// warp's mean, in one exchange through shared memory.  A row whose mean is far above its deviation loses nothing to
// cancellation: a pivot's distance from the mean is itself part of the deviation.
//
// The gradients' column sums (dgate, dscale, dshift) are kept in registers over a run of rows and written as
// one fp32 partial per (run, segment, team) to slot (run + segment) teams + team: along the stream run and segment
// only grow and one of them does, so no two meet in a slot.  A second kernel adds the slots of a segment in order, a third one
// forms dw_post and dw_pre from the per-segment sums (sum_t dr' gate yhat = sum_s gate[s] sum_{t in s} dr' yhat).
#pragma once
#include <cstdint>

#include "row_ring.h"
#include "sm100_ptx.cuh"

namespace pa {

constexpr int kNormMaxHidden = 8192;
constexpr int kNormMaxStages = 8;   // rows in flight per group
constexpr int kNormMaxTile = 8;        // rows of a tile (backward): a block has 8 warps at most
constexpr int kNormMaxBwdStages = 24;  // rows in flight per block (backward)
constexpr int kNormFwdThreads = 768;  // most threads of a block (forward)

struct NormParams {
  const int32_t* cu;  // nullptr: no per-segment factors
  int32_t total, batch, hidden;
  int32_t rows_per_chunk, chunks;
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
  float* part;     // backward: [chunks + batch][teams][3][C] partial sums (A, B, S), nullptr: no sums wanted
  int32_t stages;  // rows of the ring, and bytes of one of them (all its tensors)
  int32_t row_bytes;
  int32_t* status;
  int32_t err_cu, err_timeout;
  uint64_t wait_limit_ns;
};

// A pair's register halves, named (not shifted and or-ed together).
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  return pair_of(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float pair_sum(uint64_t a) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
  return lo + hi;
}

// Eight channels as four pairs of fp32.
struct Pairs8 {
  uint64_t p[4];
};

__device__ __forceinline__ Pairs8 pairs_of_bf16(const uint4& a) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  Pairs8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v.p[i] = pair_of(w[i] << 16, w[i] & 0xffff0000u);
  return v;
}
__device__ __forceinline__ uint4 bf16_of_pairs(const Pairs8& v) {
  return make_uint4(pack_bf16x2_pair(v.p[0]), pack_bf16x2_pair(v.p[1]), pack_bf16x2_pair(v.p[2]),
                    pack_bf16x2_pair(v.p[3]));
}
// Eight channels of type fp32 or bf16 at element `at` (global or shared memory).
template <bool kF32>
__device__ __forceinline__ Pairs8 load8(const void* p, size_t at) {
  if (kF32) {
    const ulonglong2* s = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(p) + at);
    const ulonglong2 a = s[0], b = s[1];
    return Pairs8{{a.x, a.y, b.x, b.y}};
  }
  return pairs_of_bf16(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
}
// Rounds v to the type in place and stores it.
template <bool kF32>
__device__ __forceinline__ void store8(void* p, size_t at, Pairs8& v) {
  if (kF32) {
    ulonglong2* d = reinterpret_cast<ulonglong2*>(static_cast<float*>(p) + at);
    d[0] = make_ulonglong2(v.p[0], v.p[1]);
    d[1] = make_ulonglong2(v.p[2], v.p[3]);
  } else {
    const uint4 b = bf16_of_pairs(v);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = b;
    v = pairs_of_bf16(b);
  }
}
__device__ __forceinline__ Pairs8 load_param8(const void* p, size_t at, int f32) {
  return f32 ? load8<true>(p, at) : load8<false>(p, at);
}
__device__ __forceinline__ Pairs8 pairs_splat(float x) {
  const uint64_t s = pair_of(x, x);
  return Pairs8{{s, s, s, s}};
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// The exchange of a group's warps: N values per warp through shared memory, double-buffered so that one
// barrier per exchange is enough (a buffer is rewritten two exchanges later, behind the barrier between).
struct GroupLink {
  float (*buf)[32][14];  // [2][warp of the block][14]
  int warps, warp0, warp, group;  // warps of the group, its first warp in the block, own index, group index
  int width;                      // power of two >= warps
  int flip;

  // Lane i gets the values of warp i mod width, or zeros where the group has no such warp.
  template <int N>
  __device__ __forceinline__ void exchange(float (&v)[N], int lane) {
    if (warps == 1) return;
    flip ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[flip][warp0 + warp][i] = v[i];
    }
    named_bar_sync(1 + group, warps * 32);
    const int w = lane & (width - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = w < warps ? buf[flip][warp0 + w][i] : 0.f;
  }
  // Sums of N values over what `exchange` spread out, the same in every lane.
  template <int N>
  __device__ __forceinline__ void spread_sum(float (&v)[N]) const {
    for (int s = 1; s < width; s <<= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], s);
    }
  }
};

// 1 / deviation of a variance that its roundings may have left below 0.  A NaN stays one (a maximum would make it 0,
// and the row finite but for the channel that holds it): a row with a NaN, and for a layer norm with an infinity, is NaN.
__device__ __forceinline__ float rstd_of(float var, float eps) { return rsqrtf((var < 0.f ? 0.f : var) + eps); }

// The row's mean and 1 / deviation from its warps' moments, spread over the lanes by `exchange` (one warp: its own).
__device__ __forceinline__ void merge_moments(float wm, float wq, float n, const GroupLink& link, float inv_c, int kind,
                                              float eps, float& mean, float& rstd) {
  mean = 0.f;
  if (link.warps > 1) {
    if (kind == 1) {
      const float pivot = __shfl_sync(0xffffffffu, wm, 0);
      const float d = wm - pivot;  // (lanes of no warp: n = 0)
      float v[2] = {n * d, fmaf(n * d, d, wq)};
      link.spread_sum<2>(v);
      mean = pivot + v[0] * inv_c;
      wq = v[1] - v[0] * v[0] * inv_c;
    } else {
      float v[1] = {wq};
      link.spread_sum<1>(v);
      wq = v[0];
    }
  } else {
    mean = wm;
  }
  rstd = rstd_of(wq * inv_c, eps);
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

// Factors of a segment at 8 channels: g = gate w_post, a = (1 + scale) w_pre, b = shift.
__device__ __forceinline__ Pairs8 gate_factor(const NormParams& p, int32_t seg, int col) {
  Pairs8 g = pairs_splat(1.f);
  if (p.gate != nullptr) g = load_param8(p.gate, seg * p.gate_stride + col, p.param_f32);
  if (p.w_post != nullptr) {
    const Pairs8 w = load_param8(p.w_post, col, p.param_f32);
#pragma unroll
    for (int i = 0; i < 4; ++i) g.p[i] = f2_mul(g.p[i], w.p[i]);
  }
  return g;
}
__device__ __forceinline__ Pairs8 scale_factor(const NormParams& p, int32_t seg, int col) {
  Pairs8 a = pairs_splat(1.f);
  if (p.scale != nullptr) {
    const Pairs8 s = load_param8(p.scale, seg * p.scale_stride + col, p.param_f32);
#pragma unroll
    for (int i = 0; i < 4; ++i) a.p[i] = f2_add(a.p[i], s.p[i]);
  }
  if (p.w_pre != nullptr) {
    const Pairs8 w = load_param8(p.w_pre, col, p.param_f32);
#pragma unroll
    for (int i = 0; i < 4; ++i) a.p[i] = f2_mul(a.p[i], w.p[i]);
  }
  return a;
}

// The rows of a group on their way through shared memory: up to four tensors a row, copied by the group's first
// thread.  A stage is refilled behind a barrier of the group that follows every thread's reads of it.
struct RowRing {
  uint64_t* full;  // [stages]
  uint8_t* buf;
  RingPlace at;

  __device__ __forceinline__ RowRing(uint64_t* bars, uint8_t* smem, const NormParams& p, int group)
      : full(bars + group * kNormMaxStages), buf(smem + static_cast<size_t>(group) * p.stages * p.row_bytes) {}
  // copies `row` of the given tensors (bytes b0 .. b3 a row; 0: not there) into stage s
  __device__ __forceinline__ void fill(const NormParams& p, int s, int64_t row, const void* t0, uint32_t b0,
                                       const void* t1, uint32_t b1, const void* t2, uint32_t b2, const void* t3,
                                       uint32_t b3) {
    mbar_arrive_expect_tx(full + s, p.row_bytes);
    uint8_t* dst = buf + static_cast<size_t>(s) * p.row_bytes;
    const void* src[4] = {t0, t1, t2, t3};
    const uint32_t bytes[4] = {b0, b1, b2, b3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (bytes[i] == 0) continue;
      bulk_load(dst, static_cast<const uint8_t*>(src[i]) + row * bytes[i], bytes[i], full + s);
      dst += bytes[i];
    }
  }
  // the r-th row from the current one: its wait, and where it lies
  __device__ __forceinline__ bool wait(const NormParams& p, int r, const WaitCtl& wc) const {
    return mbar_wait(full + at.stage_of(p.stages, r), at.phase_of(p.stages, r), wc);
  }
  __device__ __forceinline__ uint8_t* row(const NormParams& p, int r) const {
    return buf + static_cast<size_t>(at.stage_of(p.stages, r)) * p.row_bytes;
  }
};

// Waits, within a limit each, for the copies of the m rows from the current one on.  (Out of line: only after a timeout.)
__device__ __noinline__ void drain_rows(uint64_t* full, RingPlace at, int stages, int m, uint64_t limit_ns) {
  for (int r = 0; r < m; ++r) drain_wait(full + at.stage_of(stages, r), at.phase_of(stages, r), limit_ns);
}

// Where a group stands in its run of rows: the segment, and how far it reaches.
struct RunCursor {
  int32_t seg;
  int64_t seg_end;
  bool fresh;  // the segment has just begun
  __device__ __forceinline__ void find(const NormParams& p, int64_t row) {
    while (p.cu != nullptr && seg + 1 < p.batch && row >= p.cu[seg + 1]) ++seg;
    seg_end = p.cu != nullptr && seg + 1 < p.batch ? p.cu[seg + 1] : p.total;
    fresh = true;
  }
};

// ---------------------------------------------------------------- forward
//
// What bounds it once the loads run ahead is the number of instructions: at HBM's rate an SM has about 25 for a
// channel of a bf16 join, and shuffles, exchanges and barriers cost the same whether a warp holds 256 channels or
// 2048.  So one warp takes a whole row (kW of them where rows are long), and everything lives in shared memory: the
// row's tensors as they arrived, r over x once it is formed, and the segment's factors for all warps of the block.
// A block (one per SM) takes a run of rows; its groups take them in turn, each with a ring of its own.
struct NormFwdParams {
  NormParams n;
  int32_t groups;         // of kW warps
  int32_t ring_offset;    // bytes: the rings behind the factors
};

// A warp's 256 channels from `base` on (fewer at the row's end) lie in two halves of h = 128, each lane holding 4
// neighbours of either: fp32 values are then read and written 16 bytes a lane without bank conflicts (8 neighbours a
// lane would meet every bank twice), bf16 values 8 bytes a lane.
template <bool kF32>
__device__ __forceinline__ Pairs8 load_halves(const void* p, int64_t c, int h) {
  Pairs8 v;
  if (kF32) {
    const float* s = static_cast<const float*>(p) + c;
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s), b = *reinterpret_cast<const ulonglong2*>(s + h);
    v.p[0] = a.x;
    v.p[1] = a.y;
    v.p[2] = b.x;
    v.p[3] = b.y;
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(p) + c;
    const uint2 a = *reinterpret_cast<const uint2*>(s), b = *reinterpret_cast<const uint2*>(s + h);
    v = pairs_of_bf16(make_uint4(a.x, a.y, b.x, b.y));
  }
  return v;
}
template <bool kF32>
__device__ __forceinline__ void store_halves(void* p, size_t c, int h, const Pairs8& v) {
  if (kF32) {
    float* d = static_cast<float*>(p) + c;
    *reinterpret_cast<ulonglong2*>(d) = make_ulonglong2(v.p[0], v.p[1]);
    *reinterpret_cast<ulonglong2*>(d + h) = make_ulonglong2(v.p[2], v.p[3]);
  } else {
    uint16_t* d = static_cast<uint16_t*>(p) + c;
    const uint4 b = bf16_of_pairs(v);
    *reinterpret_cast<uint2*>(d) = make_uint2(b.x, b.y);
    *reinterpret_cast<uint2*>(d + h) = make_uint2(b.z, b.w);
  }
}

// Sum and pivoted square sum of a warp's channels of one row; `first` of them in its first sweep.
struct Moments {
  float pivot, s, q;
  __device__ __forceinline__ void start(float sum8, bool valid, float first) {
    pivot = warp_sum(valid ? sum8 : 0.f) / first;
    s = q = 0.f;
  }
  __device__ __forceinline__ void add(const Pairs8& v) {
    const uint64_t neg = pair_of(-pivot, -pivot);
    uint64_t t = 0, u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t d = f2_add(v.p[i], neg);
      u = f2_add(u, d);
      t = f2_fma(d, d, t);
    }
    s += pair_sum(u);
    q += pair_sum(t);
  }
  __device__ __forceinline__ void add_squares(const Pairs8& v) {
    uint64_t t = f2_mul(v.p[0], v.p[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) t = f2_fma(v.p[i], v.p[i], t);
    q += pair_sum(t);
  }
};

__device__ __forceinline__ float pairs_sum(const Pairs8& v) {
  const uint64_t t = f2_add(f2_add(v.p[0], v.p[1]), f2_add(v.p[2], v.p[3]));
  return pair_sum(t);
}

template <bool kF32, int kW>
__global__ void __launch_bounds__(kNormFwdThreads, 1) block_norm_fwd_kernel(const __grid_constant__ NormFwdParams fp) {
  const NormParams& p = fp.n;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[2][32][14];
  __shared__ uint64_t bars[kNormFwdThreads / 32 * kNormMaxStages];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int group = w / kW, warp = w - group * kW;
  const int C = p.hidden;
  if (threadIdx.x < fp.groups * kNormMaxStages) {
    mbar_init(bars + threadIdx.x, 1);
    fence_mbar_init();  // covers this thread's own
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  if (blockIdx.x == 0 && p.cu != nullptr) check_cu(p.cu, p.batch, p.total, p.status, p.err_cu);
  const WaitCtl wc{&abort_flag, p.status, p.wait_limit_ns, p.err_timeout};
  GroupLink link;
  link.buf = buf;
  link.warps = kW;
  link.warp0 = group * kW;
  link.warp = warp;
  link.group = group;
  link.width = kW;
  link.flip = 0;
  const bool join = p.y != nullptr;
  const uint32_t wide = static_cast<uint32_t>(C) * (kF32 ? 4 : 2), narrow = static_cast<uint32_t>(C) * 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_chunk;
  const int64_t row1 = min(row0 + p.rows_per_chunk, static_cast<int64_t>(p.total));
  float* fg = reinterpret_cast<float*>(smem);  // factors of the segment: gate w_post, (1 + scale) w_pre, shift
  float* fa = fg + C;
  float* fb = fa + C;
  RowRing ring(bars, smem + fp.ring_offset, p, group);
  bool issuing = warp == 0 && lane == 0;  // the group's copies; no longer once its wait has given up
  auto fill = [&](int s, int64_t row) {
    ring.fill(p, s, row, p.x, wide, p.y, join ? narrow : 0u, nullptr, 0u, nullptr, 0u);
  };
  int64_t row = row0 + group;  // the group's next row
  auto drain = [&](int m) { drain_rows(ring.full, ring.at, p.stages, m, p.wait_limit_ns); };
  if (issuing) ring_start(p.stages, row, fp.groups, row1, fill);

  constexpr int kStep = kW * 256;
  // f(c, h) for the lane's channels, sweep by sweep
  auto sweep = [&](auto f) {
    int base = warp * 256;
#pragma unroll 4
    for (; base + 256 <= C; base += kStep) f(base + lane * 4, 128);
    if (base < C) {  // the row's short end
      const int h = (C - base) >> 1;
      if (lane * 4 < h) f(base + lane * 4, h);
    }
  };
  // channels of this warp, in its first sweep and in all; and (lane w of kW) of warp w in all
  auto channels = [&](int wp) {
    int n = 0;
    for (int c = wp * 256; c < C; c += kStep) n += min(256, C - c);
    return static_cast<float>(n);
  };
  const float first = fmaxf(1.f, static_cast<float>(min(256, C - warp * 256)));
  const int h0 = min(128, max(0, C - warp * 256) >> 1), c0 = warp * 256 + lane * 4;
  const bool has0 = lane * 4 < h0;
  const float mine = fmaxf(1.f, channels(warp)), spread = channels(lane & (kW - 1));
  const float inv_c = 1.f / static_cast<float>(C);
  const uint64_t res2 = pair_of(p.res, p.res);
  auto finish = [&](const Moments& m, int kind, float& mean, float& rstd) {
    float v[2];
    const float q = warp_sum(m.q);
    v[0] = 0.f;
    v[1] = q;
    if (kind == 1) {
      const float s = warp_sum(m.s), d = s / mine;
      v[0] = m.pivot + d;
      v[1] = q - s * d;
    }
    link.exchange<2>(v, lane);
    merge_moments(v[0], v[1], spread, link, inv_c, kind, p.eps, mean, rstd);
  };

  RunCursor at_seg;
  at_seg.seg = p.cu != nullptr ? segment_of(p.cu, p.batch, static_cast<int32_t>(row0), lane) : 0;
  for (int64_t span = row0; span < row1;) {
    // the factors of the segment that the run is in, for all groups
    at_seg.find(p, span);
    for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
      Pairs8 f = gate_factor(p, at_seg.seg, c);
      store8<true>(fg, c, f);
      f = scale_factor(p, at_seg.seg, c);
      store8<true>(fa, c, f);
      f = p.shift != nullptr ? load_param8(p.shift, at_seg.seg * p.shift_stride + c, p.param_f32) : pairs_splat(0.f);
      store8<true>(fb, c, f);
    }
    __syncthreads();
    span = min(at_seg.seg_end, row1);
    for (; row < span; row += fp.groups) {
      // a copy that does not come within the limit is recorded; the rows are then worked on as they lie, so that the
      // barriers still meet
      ring.wait(p, 0, wc);
      const bool landed = *wc.abort_flag == 0;  // (a wait that gives up raises the flag, or has found it raised)
      uint8_t* rows = ring.row(p, 0);
      const size_t at = static_cast<size_t>(row) * C;
      Moments m;
      float mean = 0.f, rstd = 1.f;
      if (join) {
        if (p.post != 0) {
          m.start(0.f, false, 1.f);
          if (p.post == 1) {
            m.start(has0 ? pairs_sum(load_halves<false>(rows + wide, c0, h0)) : 0.f, has0, first);
            sweep([&](int c, int h) { m.add(load_halves<false>(rows + wide, c, h)); });
          } else {
            sweep([&](int c, int h) { m.add_squares(load_halves<false>(rows + wide, c, h)); });
          }
          finish(m, p.post, mean, rstd);
        }
        const uint64_t r2 = pair_of(rstd, rstd), m2 = pair_of(-mean, -mean);
        sweep([&](int c, int h) {
          Pairs8 x = load_halves<kF32>(rows, c, h);
          const Pairs8 y = load_halves<false>(rows + wide, c, h), g = load_halves<true>(fg, c, h);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x.p[i] = f2_fma(res2, x.p[i], f2_mul(g.p[i], f2_mul(f2_add(y.p[i], m2), r2)));
          store_halves<kF32>(p.r, at + c, h, x);
          if (p.pre != 0) store_halves<kF32>(rows, c, h, x);  // read back by this thread alone
        });
      }
      if (p.pre != 0) {
        m.start(0.f, false, 1.f);
        if (p.pre == 1) {
          m.start(has0 ? pairs_sum(load_halves<kF32>(rows, c0, h0)) : 0.f, has0, first);
          sweep([&](int c, int h) { m.add(load_halves<kF32>(rows, c, h)); });
        } else {
          sweep([&](int c, int h) { m.add_squares(load_halves<kF32>(rows, c, h)); });
        }
        finish(m, p.pre, mean, rstd);
        const uint64_t r2 = pair_of(rstd, rstd), m2 = pair_of(-mean, -mean);
        sweep([&](int c, int h) {
          Pairs8 x = load_halves<kF32>(rows, c, h);
          const Pairs8 a = load_halves<true>(fa, c, h), b = load_halves<true>(fb, c, h);
#pragma unroll
          for (int i = 0; i < 4; ++i) x.p[i] = f2_fma(f2_mul(f2_add(x.p[i], m2), r2), a.p[i], b.p[i]);
          store_halves<false>(p.z, at + c, h, x);
        });
      }
      // the stage is the copies' again: every thread is done with it, and what it wrote there comes before them
      fence_proxy_async_smem();
      if (kW == 1) __syncwarp();
      else named_bar_sync(1 + group, kW * 32);
      if (issuing) issuing = ring_refill(ring.at, p.stages, row, fp.groups, 1, row1, landed, fill, drain);
      ring.at.advance(p.stages, 1);
    }
    __syncthreads();  // the factors' readers are done
  }
}

// ---------------------------------------------------------------- backward
//
// A block takes a run of rows, a tile of a few at a time, in two phases.  First the rows: kW warps a row form its
// statistics and the means that the norms' gradients subtract, in sweeps over the row in shared memory (few warps a
// row, for the reason above).  Then the columns: each thread owns 8 channels (kG times 8), with the segment's factors
// and the three column sums in registers, and goes down the tile writing dx and dy.  Teams of threads share a tile's
// rows where the channels need fewer threads than a block has.
struct NormBwdParams {
  NormParams n;
  int32_t tile;           // rows of a tile, at most
  int32_t row_warps;      // warps a row in the first phase (tile * row_warps <= warps of the block)
  int32_t teams, team_warps;
  int32_t ring_offset;
};

// One row of the first phase.  With d = r - pivot and e = y - pivot (the pivots of layer norms: the mean of the row's
// first 256 channels; rms: 0), f = dz (1 + scale) w_pre and g = gate w_post, everything that the two norms' gradients
// subtract follows from sums of products of d, e, f, g and dr, so one sweep and one exchange do:
//     mean, rstd of r from sum d, sum d^2;  c0 = sum f / C,  c1 = rstd (sum f d - delta sum f) / C,  delta = mean - pivot;
//     h = g dr' = g (dr + rstd (f - c0 - rstd (d - delta) c1)), whose sum and product with yhat are linear in
//     sum g dr, g f, g, g d and in the sums of these times e.
// The sums are fp32 pairs; the differences they enter are of the size of their terms (d and e are around 0).
template <bool kF32>
struct BackRow {
  const uint8_t *r, *dz, *dr, *y;  // in shared memory (dr may be nullptr)
  const float *fa, *fg;
  int C, from, step, lane;

  template <bool kWide>
  __device__ __forceinline__ float pivot(const void* v) const {
    const int h = min(128, C >> 1);
    const bool has = lane * 4 < h;
    const float s = warp_sum(has ? pairs_sum(load_halves<kWide>(v, lane * 4, h)) : 0.f);
    return s / static_cast<float>(2 * h);
  }

  template <bool kFront, bool kBehind, bool kLayerBehind>
  __device__ __forceinline__ void means(const NormParams& p, GroupLink& link, float inv_c, float4 (&out)[2]) const {
    const float pr = kFront && p.pre == 1 ? pivot<kF32>(r) : 0.f;
    const float py = kLayerBehind ? pivot<false>(y) : 0.f;
    const uint64_t npr = pair_of(-pr, -pr), npy = pair_of(-py, -py);
    // front: 0 d, 1 d^2, 2 f, 3 f d;  behind: 4 e^2, 5 g dr e, 6 g f e, 7 g e, 8 g d e;  layer behind: 9 e, 10 g dr,
    // 11 g f, 12 g, 13 g d
    uint64_t t[14];
#pragma unroll
    for (int i = 0; i < 14; ++i) t[i] = 0;
    auto add = [&](int c, int h) {
      Pairs8 d, f, e, q, g;
      if (kFront) {
        d = load_halves<kF32>(r, c, h);
        f = load_halves<false>(dz, c, h);
        const Pairs8 a = load_halves<true>(fa, c, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d.p[i] = f2_add(d.p[i], npr);
          f.p[i] = f2_mul(f.p[i], a.p[i]);
          t[0] = f2_add(t[0], d.p[i]);
          t[1] = f2_fma(d.p[i], d.p[i], t[1]);
          t[2] = f2_add(t[2], f.p[i]);
          t[3] = f2_fma(f.p[i], d.p[i], t[3]);
        }
      }
      if (kBehind) {
        e = load_halves<false>(y, c, h);
        g = load_halves<true>(fg, c, h);
        q = dr != nullptr ? load_halves<kF32>(dr, c, h) : pairs_splat(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kLayerBehind) e.p[i] = f2_add(e.p[i], npy);
          t[4] = f2_fma(e.p[i], e.p[i], t[4]);
          const uint64_t ge = f2_mul(g.p[i], e.p[i]);
          t[5] = f2_fma(q.p[i], ge, t[5]);
          if (kFront) {
            t[6] = f2_fma(f.p[i], ge, t[6]);
            t[7] = f2_add(t[7], ge);
            t[8] = f2_fma(d.p[i], ge, t[8]);
          }
          if (kLayerBehind) {
            t[9] = f2_add(t[9], e.p[i]);
            t[10] = f2_fma(q.p[i], g.p[i], t[10]);
            if (kFront) {
              t[11] = f2_fma(f.p[i], g.p[i], t[11]);
              t[12] = f2_add(t[12], g.p[i]);
              t[13] = f2_fma(d.p[i], g.p[i], t[13]);
            }
          }
        }
      }
    };
    int base = from;
#pragma unroll(kBehind ? 1 : 2)
    for (; base + 256 <= C; base += step) add(base + lane * 4, 128);
    if (base < C) {  // the row's short end
      const int h = (C - base) >> 1;
      if (lane * 4 < h) add(base + lane * 4, h);
    }
    float v[14];
#pragma unroll
    for (int i = 0; i < 14; ++i) {
      const bool used = i < 4 ? kFront : i < 6 ? kBehind : i < 9 ? kBehind && kFront : i < 11 ? kLayerBehind : kLayerBehind && kFront;
      v[i] = used ? warp_sum(pair_sum(t[i])) : 0.f;
    }
    link.exchange<14>(v, lane);
    if (link.warps > 1) link.spread_sum<14>(v);
    float mean_r = 0.f, rstd_r = 1.f, delta = 0.f, c0 = 0.f, c1 = 0.f;
    if (kFront) {
      if (p.pre == 1) {
        delta = v[0] * inv_c;
        mean_r = pr + delta;
      }
      rstd_r = rstd_of(v[1] * inv_c - delta * delta, p.eps);
      c0 = p.pre == 1 ? v[2] * inv_c : 0.f;
      c1 = rstd_r * (v[3] - delta * v[2]) * inv_c;
    }
    out[0] = make_float4(mean_r, rstd_r, c0, c1);
    if (kBehind) {
      const float shift = kLayerBehind ? v[9] * inv_c : 0.f;
      const float rstd_y = rstd_of(v[4] * inv_c - shift * shift, p.eps);
      const float k = rstd_r * c1;
      const float sum_he = kFront ? v[5] + rstd_r * (v[6] - c0 * v[7] - k * (v[8] - delta * v[7])) : v[5];
      float e0 = 0.f, sum_h = 0.f;
      if (kLayerBehind) {
        sum_h = kFront ? v[10] + rstd_r * (v[11] - c0 * v[12] - k * (v[13] - delta * v[12])) : v[10];
        e0 = sum_h * inv_c;
      }
      out[1] = make_float4(py + shift, rstd_y, e0, rstd_y * (sum_he - shift * sum_h) * inv_c);
    }
  }
};

template <bool kF32, int kG>
__global__ void __launch_bounds__(256, kG == 1 ? 2 : 1)
    block_norm_bwd_kernel(const __grid_constant__ NormBwdParams bp) {
  const NormParams& p = bp.n;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[2][32][14];
  __shared__ float4 scalars[kNormMaxTile][2];  // per row: mean, rstd, c0, c1 of the norm in front, and of the one behind
  __shared__ uint64_t bars[kNormMaxBwdStages];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int C = p.hidden;
  if (threadIdx.x < p.stages) {
    mbar_init(bars + threadIdx.x, 1);
    fence_mbar_init();  // covers this thread's own
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  if (blockIdx.x == 0 && p.cu != nullptr) check_cu(p.cu, p.batch, p.total, p.status, p.err_cu);
  const WaitCtl wc{&abort_flag, p.status, p.wait_limit_ns, p.err_timeout};
  const bool join = p.y != nullptr, front = p.dz != nullptr, given = p.dr != nullptr;
  const bool normed = join && p.post != 0;
  const uint32_t wide = static_cast<uint32_t>(C) * (kF32 ? 4 : 2), narrow = static_cast<uint32_t>(C) * 2;
  const uint32_t br = front ? wide : 0u, bz = front ? narrow : 0u, bd = given ? wide : 0u, by = join ? narrow : 0u;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_chunk;
  const int64_t row1 = min(row0 + p.rows_per_chunk, static_cast<int64_t>(p.total));
  const float inv_c = 1.f / static_cast<float>(C);
  float* fg = reinterpret_cast<float*>(smem);  // factors of the segment: gate w_post, (1 + scale) w_pre
  float* fa = fg + C;
  RowRing ring(bars, smem + bp.ring_offset, p, 0);
  auto fill = [&](int s, int64_t row) { ring.fill(p, s, row, p.x, br, p.dz, bz, p.dr, bd, p.y, by); };
  auto drain = [&](int m) { drain_rows(ring.full, ring.at, p.stages, m, p.wait_limit_ns); };
  if (threadIdx.x == 0) ring_start(p.stages, row0, 1, row1, fill);

  // first phase: group of row_warps warps
  GroupLink link;
  link.buf = buf;
  link.warps = link.width = bp.row_warps;
  link.group = w / bp.row_warps;
  link.warp0 = link.group * bp.row_warps;
  link.warp = w - link.warp0;
  link.flip = 0;
  const int step = bp.row_warps * 256, from = link.warp * 256;

  // second phase: team, and the thread's channels
  const int team = w / bp.team_warps, team_warp = w - team * bp.team_warps;
  int col[kG], half[kG];
  bool own[kG];
#pragma unroll
  for (int k = 0; k < kG; ++k) {
    const int base = (team_warp + k * bp.team_warps) * 256;
    half[k] = min(128, max(0, C - base) >> 1);
    col[k] = base + lane * 4;
    own[k] = team < bp.teams && lane * 4 < half[k];
  }
  Pairs8 sa[kG], sb[kG], ss[kG], g[kG], a[kG];
#pragma unroll
  for (int k = 0; k < kG; ++k) sa[k] = sb[k] = ss[k] = pairs_splat(0.f);
  const uint64_t res2 = pair_of(p.res, p.res);
  auto flush = [&](int32_t s) {
    if (p.part == nullptr) return;
    float* dst = p.part + ((static_cast<size_t>(blockIdx.x) + s) * bp.teams + team) * 3 * C;
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      if (!own[k]) continue;
      if (join) store_halves<true>(dst, col[k], half[k], sa[k]);
      if (front) {
        store_halves<true>(dst + C, col[k], half[k], sb[k]);
        store_halves<true>(dst + 2 * static_cast<size_t>(C), col[k], half[k], ss[k]);
      }
    }
  };
  RunCursor at_seg;
  at_seg.seg = p.cu != nullptr ? segment_of(p.cu, p.batch, static_cast<int32_t>(row0), lane) : 0;
  at_seg.find(p, row0);
  for (int64_t row = row0; row < row1;) {
    if (row >= at_seg.seg_end) {
      flush(at_seg.seg);
      at_seg.find(p, row);
#pragma unroll
      for (int k = 0; k < kG; ++k) sa[k] = sb[k] = ss[k] = pairs_splat(0.f);
    }
    if (at_seg.fresh) {  // (the last tile's readers are behind its closing barrier)
      at_seg.fresh = false;
      for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
        Pairs8 f = gate_factor(p, at_seg.seg, c);
        store8<true>(fg, c, f);
        f = scale_factor(p, at_seg.seg, c);
        store8<true>(fa, c, f);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kG; ++k) {
        if (!own[k]) continue;
        g[k] = load_halves<true>(fg, col[k], half[k]);
        a[k] = load_halves<true>(fa, col[k], half[k]);
      }
    }
    const int n = static_cast<int>(min(static_cast<int64_t>(bp.tile), min(at_seg.seg_end, row1) - row));

    if (link.group < n) ring.wait(p, link.group, wc);  // as in the forward kernel
    if (link.group < n && (front || normed)) {
      const int r = link.group;
      const uint8_t* src = ring.row(p, r);
      const BackRow<kF32> x{src, src + br, given ? src + br + bz : nullptr, src + br + bz + bd, fa, fg, C, from, step, lane};
      float4 out[2];
      if (!normed) x.template means<true, false, false>(p, link, inv_c, out);
      else if (!front && p.post == 1) x.template means<false, true, true>(p, link, inv_c, out);
      else if (!front) x.template means<false, true, false>(p, link, inv_c, out);
      else if (p.post == 1) x.template means<true, true, true>(p, link, inv_c, out);
      else x.template means<true, true, false>(p, link, inv_c, out);
      if (link.warp == 0 && lane == 0) {
        scalars[r][0] = out[0];
        scalars[r][1] = out[1];
      }
    }
    __syncthreads();
    // every row of the tile has been waited for; the flag is up if one has not come
    const bool landed = *wc.abort_flag == 0;
    for (int r = team; r < n; r += bp.teams) {
      const uint8_t* src = ring.row(p, r);
      uint8_t* dx = static_cast<uint8_t*>(p.r) + (row + r) * static_cast<int64_t>(wide);
      uint8_t* dy = static_cast<uint8_t*>(p.z) + (row + r) * static_cast<int64_t>(narrow);
      const float4 sr = scalars[r][0], sy = scalars[r][1];
      const uint64_t mr2 = pair_of(-sr.x, -sr.x), r2 = pair_of(sr.y, sr.y), n0 = pair_of(-sr.z, -sr.z),
                     n1 = pair_of(-sr.w, -sr.w);
      const uint64_t my2 = pair_of(-sy.x, -sy.x), y2 = pair_of(sy.y, sy.y), e0 = pair_of(-sy.z, -sy.z),
                     e1 = pair_of(-sy.w, -sy.w);
#pragma unroll
      for (int k = 0; k < kG; ++k) {
        if (!own[k]) continue;
        Pairs8 d = given ? load_halves<kF32>(src + br + bz, col[k], half[k]) : pairs_splat(0.f);
        if (front) {
          Pairs8 v = load_halves<kF32>(src, col[k], half[k]);
          const Pairs8 z = load_halves<false>(src + br, col[k], half[k]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v.p[i] = f2_mul(f2_add(v.p[i], mr2), r2);
            sb[k].p[i] = f2_fma(z.p[i], v.p[i], sb[k].p[i]);
            ss[k].p[i] = f2_add(ss[k].p[i], z.p[i]);
            d.p[i] = f2_fma(r2, f2_fma(v.p[i], n1, f2_fma(z.p[i], a[k].p[i], n0)), d.p[i]);
          }
        }
        Pairs8 t;
#pragma unroll
        for (int i = 0; i < 4; ++i) t.p[i] = f2_mul(res2, d.p[i]);
        store_halves<kF32>(dx, col[k], half[k], t);
        if (!join) continue;
        Pairs8 y = load_halves<false>(src + br + bz + bd, col[k], half[k]);
        if (normed) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y.p[i] = f2_mul(f2_add(y.p[i], my2), y2);
            sa[k].p[i] = f2_fma(d.p[i], y.p[i], sa[k].p[i]);
            d.p[i] = f2_mul(y2, f2_fma(y.p[i], e1, f2_fma(d.p[i], g[k].p[i], e0)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sa[k].p[i] = f2_fma(d.p[i], y.p[i], sa[k].p[i]);
            d.p[i] = f2_mul(d.p[i], g[k].p[i]);
          }
        }
        store_halves<false>(dy, col[k], half[k], d);
      }
    }
    __syncthreads();  // the tile's stages, scalars and factors are free
    // (that the copies have been drained is kept in the flag, not by thread, for the registers)
    if (threadIdx.x == 0 && (landed || *wc.abort_flag != 2) &&
        !ring_refill(ring.at, p.stages, row, 1, n, row1, landed, fill, drain))
      *wc.abort_flag = 2;
    ring.at.advance(p.stages, n);
    row += n;
  }
  flush(at_seg.seg);
}

struct NormSumParams {
  const int32_t* cu;  // nullptr: one segment over all tokens
  int32_t total, batch, hidden, rows_per_chunk, chunks, teams, param_f32;
  int32_t use;  // bit k: sum k (A, B, S) is needed
  int32_t long_runs;         // block_norm_sum_kernel: a segment of more runs of rows is a long one
  int32_t long_col_blocks;   // ... and takes this many blocks of each of the grid's rows
  const float* part;
  float* sums;  // [2][batch][C]: A and B of every segment, nullptr: not needed
  const void* w_post;
  const void* w_pre;
  float* dgate;   // [batch][C], each may be nullptr
  float* dscale;
  float* dshift;
};

// Adds the slots c0 + first, c0 + first + step, ... below c1 at 4 channels, for the three sums.
__device__ __forceinline__ void add_slots(const NormSumParams& p, int64_t c0, int64_t c1, int first, int step, int col,
                                          float4 (&t)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) t[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int64_t c = c0 + first; c < c1; c += step) {
    const float* src = p.part + static_cast<size_t>(c) * 3 * p.hidden + col;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (!(p.use >> k & 1)) continue;
      const float4 v = *reinterpret_cast<const float4*>(src + static_cast<size_t>(k) * p.hidden);
      t[k].x += v.x;
      t[k].y += v.y;
      t[k].z += v.z;
      t[k].w += v.w;
    }
  }
}

// The slots of segment s.
__device__ __forceinline__ void slots_of(const NormSumParams& p, int32_t s, int64_t& c0, int64_t& c1) {
  c0 = c1 = 0;
  const int32_t beg = p.cu != nullptr ? p.cu[s] : 0, end = p.cu != nullptr ? p.cu[s + 1] : p.total;
  if (beg >= 0 && end > beg && end <= p.total) {  // (cu_seqlens may be bad)
    c0 = (static_cast<int64_t>(beg / p.rows_per_chunk) + s) * p.teams;
    c1 = (static_cast<int64_t>(min((end - 1) / p.rows_per_chunk + 1, p.chunks)) + s) * p.teams;
  }
}

// Writes sum k of segment s at 4 channels: the raw sum where the weights' gradients need it, and the output.  A segment
// without tokens (`some` false) gets 0 whatever the weight is.
__device__ __forceinline__ void put_sum(const NormSumParams& p, int32_t s, int k, int col, float4 t, bool some) {
  const size_t at = static_cast<size_t>(s) * p.hidden + col;
  if (k < 2 && p.sums != nullptr)
    *reinterpret_cast<float4*>(p.sums + static_cast<size_t>(k) * p.batch * p.hidden + at) = t;
  float* out = k == 0 ? p.dgate : k == 1 ? p.dscale : p.dshift;
  if (out == nullptr) return;
  const void* weight = k == 0 ? p.w_post : k == 1 ? p.w_pre : nullptr;
  float f[4] = {t.x, t.y, t.z, t.w};
  if (weight != nullptr && some) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] *= p.param_f32 ? static_cast<const float*>(weight)[col + i]
                          : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(weight)[col + i]) << 16);
  }
  *reinterpret_cast<float4*>(out + at) = make_float4(f[0], f[1], f[2], f[3]);
}

// Per segment: the sum of its slots.  Where there are many segments a thread takes 4 channels of one, slot after slot (a
// short image has one or two).  A long one among them would keep a few threads busy for the whole call (602 us for one
// of 65536 tokens and 40 of 200, 256 channels; 168 us as it is), so its channels go 32 a block to blocks of
// their own behind those of the segments, the slots 32 apart and the 32 parts added in order.  A segment of more than
// long_runs runs holds the first row of a run whose number is a multiple of long_runs; the first such row names it, and
// block j of these looks for its segment there.
constexpr int kNormSumThreads = 256;
__global__ void __launch_bounds__(kNormSumThreads) block_norm_sum_kernel(const __grid_constant__ NormSumParams p) {
  pdl_wait_primary();
  __shared__ float4 acc[3][32][8];
  int64_t c0, c1;
  float4 t[3];
  const int64_t most = static_cast<int64_t>(p.long_runs) * p.teams;  // slots
  if (blockIdx.x < p.batch) {
    const int col = (blockIdx.y * kNormSumThreads + threadIdx.x) * 4;
    const int32_t s = blockIdx.x;
    slots_of(p, s, c0, c1);
    if (col >= p.hidden || c1 - c0 > most) return;
    add_slots(p, c0, c1, 0, 1, col, t);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (p.use >> k & 1) put_sum(p, s, k, col, t[k], c1 > c0);
    return;
  }
  const int32_t j = (blockIdx.x - p.batch) / p.long_col_blocks, rest = (blockIdx.x - p.batch) - j * p.long_col_blocks;
  const int64_t stride = static_cast<int64_t>(p.long_runs) * p.rows_per_chunk, row = j * stride;
  const int32_t s = segment_of(p.cu, p.batch, static_cast<int32_t>(row), threadIdx.x & 31);
  slots_of(p, s, c0, c1);
  if (c1 - c0 <= most || (p.cu[s] + stride - 1) / stride != j) return;
  const int lane = threadIdx.x & 7, part = threadIdx.x >> 3;
  const int col = (rest * gridDim.y + blockIdx.y) * 32 + lane * 4;
  add_slots(p, c0, col < p.hidden ? c1 : c0, part, 32, col, t);
#pragma unroll
  for (int k = 0; k < 3; ++k) acc[k][part][lane] = t[k];
  __syncthreads();
  if (part >= 3 || col >= p.hidden || !(p.use >> part & 1)) return;
  float4 u = acc[part][0][lane];
#pragma unroll 8
  for (int i = 1; i < 32; ++i) {
    u.x += acc[part][i][lane].x;
    u.y += acc[part][i][lane].y;
    u.z += acc[part][i][lane].z;
    u.w += acc[part][i][lane].w;
  }
  put_sum(p, s, part, col, u, true);
}

// Where there are few segments a block takes 128 channels of one: its 32 warps take the slots 32 apart, and the warps'
// sums are added in order.
constexpr int kNormSumLongThreads = 1024;
__global__ void __launch_bounds__(kNormSumLongThreads) block_norm_sum_long_kernel(const __grid_constant__ NormSumParams p) {
  pdl_wait_primary();
  __shared__ float4 acc[3][32][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.y * 128 + lane * 4;
  const int32_t s = blockIdx.x;
  int64_t c0, c1;
  slots_of(p, s, c0, c1);
  float4 t[3];
  add_slots(p, c0, col < p.hidden ? c1 : c0, w, 32, col, t);
#pragma unroll
  for (int k = 0; k < 3; ++k) acc[k][w][lane] = t[k];
  __syncthreads();
  if (w >= 3 || col >= p.hidden || !(p.use >> w & 1)) return;
  float4 u = acc[w][0][lane];
#pragma unroll 8
  for (int j = 1; j < 32; ++j) {
    u.x += acc[w][j][lane].x;
    u.y += acc[w][j][lane].y;
    u.z += acc[w][j][lane].z;
    u.w += acc[w][j][lane].w;
  }
  put_sum(p, s, w, col, u, c1 > c0);
}

struct NormWeightParams {
  const int32_t* cu;  // nullptr: one segment over all tokens
  int32_t batch, hidden, param_f32;
  const float* sums;  // [2][batch][C]
  const void* gate;
  const void* scale;
  int64_t gate_stride, scale_stride;
  float* dw_post;
  float* dw_pre;
};

// dw_post = sum_s gate[s] A[s], dw_pre = sum_s (1 + scale[s]) B[s]: one block per 32 channels and weight, its
// 8 warps taking the segments 8 apart.  The factors of a segment without tokens are not read: rows behind a padded
// batch may hold anything, and NaN times its sum of 0 is not 0.
__global__ void __launch_bounds__(256) block_norm_weight_kernel(const __grid_constant__ NormWeightParams p) {
  pdl_wait_primary();
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
      if (p.cu != nullptr && p.cu[s + 1] <= p.cu[s]) continue;
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
