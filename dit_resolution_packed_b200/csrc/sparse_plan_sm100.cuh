// sparse_plan_sm100.cuh -- which key blocks a block of queries sees: the selection by a cheap score, and the work
// lists of the block-sparse attention kernels.
//
// A pack's blocks of 128 tokens are numbered along the stream: block b of segment s is row cu[s] / 128 + s + b of
// the tables (integer division).  cu[s] / 128 + s grows strictly with s and a segment's blocks never reach its
// successor's first row, so a row names one block, the segment of a row is found by binary search, and no table
// size has to be read back from the device.  Pairs of blocks (256) and groups of eight (1024) are numbered alike.
//
// Selection.  The score of (query block, key block) is the inner product of their mean vectors.  Means, products
// and sums are fp64.  A sum of 128 bf16 values is exact there while their exponents lie within 38 of each other; the
// division by the tokens of a short block and the products' sum round, in an order that is fixed (so a selection repeats
// itself, and equal means give equal scores).  Scores that differ by a few roundings of 64 bits may be ordered either
// way by another order of additions.  It reads q and k once (memory-bound); the scores themselves are d products per
// pair of blocks, 1/16384 of the attention's.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "sm100_ptx.cuh"

namespace pa {

constexpr int kSparseClasses = 16;  // of the work order: items of 2^(c-1) .. 2^c - 1 steps (0 steps: class 0)
constexpr int kDescInts = 12;
constexpr int kSelectMaxBlocks = 2048;  // key blocks of a segment in pa_block_select (8 rows of scores in shared memory)

// A segment of the pack and a unit (block, pair or group of 2^log2 tokens) of it; valid: the unit has tokens.
struct UnitAt {
  int32_t seg, beg, len, unit;
  bool valid;
};

// The unit of a row of a table.  Reads cu_seqlens only inside [0, batch]; a segment that does not lie in
// [0, total], or is longer than max_seqlen, has no units.
__device__ __forceinline__ UnitAt unit_at(const int32_t* cu, int32_t batch, int32_t total, int32_t max_seqlen,
                                          int64_t row, int log2) {
  int32_t lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if ((static_cast<int64_t>(__ldg(cu + mid)) >> log2) + mid <= row) lo = mid; else hi = mid;
  }
  UnitAt u;
  u.seg = lo;
  u.beg = __ldg(cu + lo);
  const int32_t end = __ldg(cu + lo + 1);
  const bool ok = u.beg >= 0 && end > u.beg && end <= total && end - u.beg <= max_seqlen;
  u.len = ok ? end - u.beg : 0;
  const int64_t first = (static_cast<int64_t>(u.beg) >> log2) + lo;
  const int64_t unit = row - first;
  u.valid = ok && unit >= 0 && unit < ((static_cast<int64_t>(u.len) + (1 << log2) - 1) >> log2);
  u.unit = u.valid ? static_cast<int32_t>(unit) : 0;
  return u;
}

// Records what is wrong with cu_seqlens (one block).
__device__ __forceinline__ void check_pack(const int32_t* cu, int32_t batch, int32_t total, int32_t max_seqlen,
                                           int32_t* status, int32_t err_cu, int32_t err_max) {
  if (threadIdx.x == 0 && (cu[0] != 0 || cu[batch] != total)) atomicCAS(status, 0, err_cu);
  for (int32_t i = threadIdx.x; i < batch; i += blockDim.x) {
    const int32_t a = cu[i], b = cu[i + 1];
    if (b < a) atomicCAS(status, 0, err_cu);
    else if (static_cast<int64_t>(b) - a > max_seqlen) atomicCAS(status, 0, err_max);
  }
}

// ---------------------------------------------------------------- selection
struct SelectParams {
  const uint16_t* x[2];  // q, k: bf16 [T, H, d]
  const int32_t* cu;
  int32_t batch, total, heads, head_dim, max_seqlen, width, min_blocks;
  double density;
  double* mean;  // [2][H][rows][d]
  int64_t rows;
  int32_t* idx;  // [H][rows][width]
  int32_t* cnt;  // [H][rows]
  int32_t* status;
  int32_t err_cu, err_max;
};

constexpr int kPoolThreads = 256;

// Means of one block of tokens over 256 channels of q (z = 0) or k (z = 1): 8 warps take 16 tokens each, a lane 8
// channels, and the warps' sums meet in shared memory.  201 MB in 46 us, DRAM and the conversions to fp64 (16 a clock
// and SM) in each other's way; all of a warp's loads at once cost occupancy (52 us), and fp64 put together from the
// bits of a bf16 with integer instructions, without conversions, took 53 us.  Four blocks an SM (64 registers, loads
// further ahead) are 3 us faster than five, eight 7 us slower.
__global__ void __launch_bounds__(kPoolThreads, 4) select_pool_kernel(const __grid_constant__ SelectParams p) {
  __shared__ double acc[8][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int which = blockIdx.z;
  const int32_t channels = p.heads * p.head_dim;
  const int32_t c0 = blockIdx.y * 256 + lane * 8;
  if (blockIdx.x == 0 && blockIdx.y == 0 && which == 0)
    check_pack(p.cu, p.batch, p.total, p.max_seqlen, p.status, p.err_cu, p.err_max);
  const UnitAt u = unit_at(p.cu, p.batch, p.total, p.max_seqlen, row, 7);
  if (!u.valid) {
    // a row that is no block: an empty list (for the heads whose first channel is among these 256)
    if (which == 0) {
      const int h0 = (blockIdx.y * 256 + p.head_dim - 1) / p.head_dim;
      const int h1 = min(p.heads, static_cast<int>((blockIdx.y * 256 + 256 + p.head_dim - 1) / p.head_dim));
      for (int h = h0; h < h1; ++h) {
        const int64_t at = static_cast<int64_t>(h) * p.rows + row;
        if (threadIdx.x == 0) p.cnt[at] = 0;
        for (int i = threadIdx.x; i < p.width; i += kPoolThreads) p.idx[at * p.width + i] = -1;
      }
    }
    return;
  }
  const int32_t tokens = min(128, u.len - u.unit * 128);
  double s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.0;
  if (c0 < channels) {
    const uint16_t* src = p.x[which] + (static_cast<size_t>(u.beg) + u.unit * 128) * channels + c0;
#pragma unroll 8
    for (int t = w; t < tokens; t += 8) {
      float v[8];
      bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(t) * channels)), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += static_cast<double>(v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[w][i * 32 + lane] = s[i];
  __syncthreads();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= channels) return;
  double t = 0.0;
  const int at = (threadIdx.x & 7) * 32 + (threadIdx.x >> 3);
#pragma unroll
  for (int i = 0; i < 8; ++i) t += acc[i][at];
  const int h = c / p.head_dim;
  p.mean[((static_cast<int64_t>(which) * p.heads + h) * p.rows + row) * p.head_dim + (c - h * p.head_dim)] = t / tokens;
}

// Monotone map of a score to an unsigned integer; a NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint64_t score_key(double s) {
  if (!(s == s)) s = -INFINITY;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
  return (b >> 63) ? ~b : (b | (1ull << 63));
}

// One block per (group of 8 query blocks, head).  Scores: a chunk of 32 key blocks at a time, each warp an eighth of the
// channels for all 8 x 32 pairs (a lane one key block and 8 sums, so a value read from shared memory serves 8
// products), the warps' parts added in order; the next chunk's means come into registers meanwhile.  Then warp w
// selects for query block w of the group.  128 blocks x 24 heads: 25 us, waiting for shared memory (40 us with a
// product a value read).
template <int D>
__global__ void __launch_bounds__(256) select_topk_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) double sm[];
  constexpr int kRow = D + 2;  // of a key block's means: 16-byte aligned, and no bank conflicts across 32 rows
  double* qs = sm;             // [8][D]
  double* ks = qs + 8 * D;     // [32][kRow]
  double* part = ks + 32 * kRow;  // [8 warps][8 query blocks][32]
  uint64_t* keys = reinterpret_cast<uint64_t*>(part + 8 * 8 * 32);  // [8][nb]
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int h = blockIdx.y;
  pdl_wait_primary();
  const UnitAt u = unit_at(p.cu, p.batch, p.total, p.max_seqlen, blockIdx.x, 10);
  if (!u.valid) return;
  const int nb = (u.len + 127) >> 7;
  const int q0 = u.unit * 8, nq = min(8, nb - q0);
  const int64_t row0 = (u.beg >> 7) + u.seg;  // of the segment's first block
  const double* qm = p.mean + (static_cast<int64_t>(h) * p.rows + row0) * D;
  const double* km = qm + static_cast<int64_t>(p.heads) * p.rows * D;
  for (int i = threadIdx.x; i < 8 * D; i += 256) qs[i] = i < nq * D ? qm[q0 * D + i] : 0.0;
  constexpr int kPer = 32 * D / 512;  // pairs of means a thread brings
  double2 next[kPer];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = (threadIdx.x + 256 * i) * 2;
      next[i] = k0 * D + at < nb * D ? *reinterpret_cast<const double2*>(km + static_cast<int64_t>(k0) * D + at)
                                     : make_double2(0.0, 0.0);
    }
  };
  fetch(0);
  for (int k0 = 0; k0 < nb; k0 += 32) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = (threadIdx.x + 256 * i) * 2;
      *reinterpret_cast<double2*>(ks + (at / D) * kRow + at % D) = next[i];
    }
    __syncthreads();
    if (k0 + 32 < nb) fetch(k0 + 32);
    double acc[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) acc[r] = 0.0;
#pragma unroll 4
    for (int c = w * (D / 8); c < (w + 1) * (D / 8); c += 2) {
      const double2 b = *reinterpret_cast<const double2*>(ks + lane * kRow + c);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const double2 a = *reinterpret_cast<const double2*>(qs + r * D + c);
        acc[r] = fma(a.x, b.x, acc[r]);
        acc[r] = fma(a.y, b.y, acc[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) part[(w * 8 + r) * 32 + lane] = acc[r];
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[(i * 8 + w) * 32 + lane];
    if (k0 + lane < nb) keys[static_cast<size_t>(w) * nb + k0 + lane] = score_key(s);
  }
  __syncwarp();
  if (w >= nq) return;
  const uint64_t* mine = keys + static_cast<size_t>(w) * nb;
  const int keep = min(nb, max(p.min_blocks, static_cast<int>(ceil(p.density * static_cast<double>(nb)))));
  // the largest threshold that at least `keep` scores reach, bit by bit from the top; done early when exactly
  // `keep` reach it
  uint64_t all = ~0ull, any = 0;  // the scores' common leading bits need no count
  for (int i = lane; i < nb; i += 32) {
    all &= mine[i];
    any |= mine[i];
  }
  const uint64_t differ =
      (static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32)) ^
                             __reduce_and_sync(0xffffffffu, static_cast<uint32_t>(all >> 32)))
       << 32) |
      (__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any)) ^
       __reduce_and_sync(0xffffffffu, static_cast<uint32_t>(all)));
  const int top = differ == 0 ? -1 : 63 - __clzll(static_cast<long long>(differ));
  uint64_t bar = top == 63 ? 0 : mine[0] >> (top + 1) << (top + 1);
  int reached = nb;
  for (int bit = top; bit >= 0 && reached != keep; --bit) {
    const uint64_t cand = bar | (1ull << bit);
    int c = 0;
    for (int i = lane; i < nb; i += 32) c += mine[i] >= cand;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= keep) {
      bar = cand;
      reached = c;
    }
  }
  // of the scores that equal the threshold, the lowest blocks are taken until `keep` are
  int above = 0;
  for (int i = lane; i < nb; i += 32) above += mine[i] > bar;
  above = __reduce_add_sync(0xffffffffu, above);
  int ties = keep - above, taken = 0;
  const int64_t at = static_cast<int64_t>(h) * p.rows + row0 + q0 + w;
  int32_t* out = p.idx + at * p.width;
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = 0; i0 < nb; i0 += 32) {
    const int i = i0 + lane;
    const uint64_t key = i < nb ? mine[i] : 0;
    const bool over = i < nb && key > bar, tie = i < nb && key == bar;
    const uint32_t mt = __ballot_sync(0xffffffffu, tie);
    const bool pick = over || (tie && __popc(mt & below) < ties);
    const uint32_t mp = __ballot_sync(0xffffffffu, pick);
    if (pick) out[taken + __popc(mp & below)] = i;
    ties -= __popc(mt);
    taken += __popc(mp);
  }
  for (int i = keep + lane; i < p.width; i += 32) out[i] = -1;
  if (lane == 0) p.cnt[at] = keep;
}

// ---------------------------------------------------------------- work lists
struct SparsePlanParams {
  CUtensorMap tmpl[4];     // q, k, v[, dout] over the whole [T, H*d] matrix
  CUtensorMap small[4];    // the same, encoded as a tensor of a row (write_part_map)
  const void* base[4];
  const int32_t* cu;
  const int32_t* idx;      // [H][rows][width]
  const int32_t* cnt;      // [H][rows]
  int32_t batch, total, heads, max_seqlen, width, n_maps;
  int64_t rows;            // block rows of the tables
  int64_t units;           // rows of the work list per head: pairs (forward) or key blocks (backward)
  uint64_t row_bytes;
  int32_t* counts;         // [0] items, [2] work counter
  int32_t* cls;            // [heads * units, rounded up to 4] class of an item, -1: none there
  int32_t* order;          // [heads * units] items, longest classes first
  int32_t* desc;           // [heads * units][kDescInts]
  int2* steps;             // forward: [heads * units][width]
  uint32_t* bits;          // backward: [heads][rows][words] query blocks that name a key block, zeroed before
  int32_t words;
  uint8_t* maps;           // [batch][n_maps] tensor maps
  int32_t sorted;          // 0: items are taken as they lie (no classes, no order)
  int32_t* status;
  int32_t err_cu, err_max, err_blocks;
};

// The tensor maps of segment `seg`: the templates with base and row extent moved, so that a tile's rows past the
// segment read zeros and nothing of a neighbouring image (whatever it holds) enters a product.  Warp `seg` of a plan
// writes them (a work list has at least a row per segment), not the one that finds the segment's first unit: with
// cu_seqlens that decrease, that row may be found to be another segment's, and later units of this one still exist.
__device__ __forceinline__ void write_maps(const SparsePlanParams& p, int64_t seg, int lane) {
  if (seg >= p.batch || lane >= p.n_maps) return;
  const int32_t beg = __ldg(p.cu + seg), end = __ldg(p.cu + seg + 1);
  if (beg < 0 || end <= beg || end > p.total) return;  // no units
  uint8_t* dst = p.maps + (static_cast<size_t>(seg) * p.n_maps + lane) * 128;
  write_part_map<1>(dst, p.tmpl[lane], p.small[lane], static_cast<uint64_t>(end - beg) * p.row_bytes,
                    static_cast<const uint8_t*>(p.base[lane]) + static_cast<uint64_t>(beg) * p.row_bytes,
                    static_cast<uint32_t>(end - beg));
  fence_tmap_release();
}

// Length of a block's list, 0 (and the status recorded) if it is not an increasing list of the segment's blocks.
__device__ __forceinline__ int32_t checked_list(const SparsePlanParams& p, int64_t at, int32_t nb, int lane) {
  const int32_t n = __ldg(p.cnt + at);
  bool bad = n < 0 || n > p.width;
  const int32_t m = bad ? 0 : n;
  const int32_t* list = p.idx + at * p.width;
  for (int32_t i = lane; i < m; i += 32) {
    const int32_t v = __ldg(list + i);
    bad |= v < 0 || v >= nb || (i > 0 && __ldg(list + i - 1) >= v);
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) atomicCAS(p.status, 0, p.err_blocks);
    return 0;
  }
  return m;
}

__device__ __forceinline__ bool in_list(const int32_t* list, int32_t n, int32_t v) {
  int32_t lo = 0, hi = n;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (__ldg(list + mid) < v) lo = mid + 1; else hi = mid;
  }
  return lo < n && __ldg(list + lo) == v;
}

__device__ __forceinline__ void file_item(const SparsePlanParams& p, int64_t item, int32_t steps) {
  if (p.sorted) p.cls[item] = min(kSparseClasses - 1, 32 - __clz(steps));
}

// Forward: one warp per (head, pair of query blocks).  The two lists become one list of steps: first the blocks
// that both name (their K and V tiles are loaded once for both query tiles), then the others side by side, so both
// tiles stay busy in every step but the last few and tile t is busy exactly in steps [0, cnt_t).
__global__ void __launch_bounds__(128) sparse_plan_fwd_kernel(const __grid_constant__ SparsePlanParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    check_pack(p.cu, p.batch, p.total, p.max_seqlen, p.status, p.err_cu, p.err_max);
    if (!p.sorted && threadIdx.x == 0) {
      p.counts[0] = static_cast<int32_t>(p.units * p.heads);
      p.counts[2] = 0;
    }
  }
  write_maps(p, item, lane);
  if (item >= p.units * p.heads) return;
  const int32_t h = static_cast<int32_t>(item / p.units);
  const UnitAt u = unit_at(p.cu, p.batch, p.total, p.max_seqlen, item - h * p.units, 8);
  int32_t* d = p.desc + item * kDescInts;
  if (!u.valid) {
    if (lane == 0) {
      d[0] = -1;
      if (p.sorted) p.cls[item] = -1;
    }
    return;
  }
  const int32_t nb = (u.len + 127) >> 7;
  const bool two = u.unit * 256 + 128 < u.len;
  const int64_t at0 = static_cast<int64_t>(h) * p.rows + (u.beg >> 7) + u.seg + 2 * u.unit;
  const int32_t* l0 = p.idx + at0 * p.width;
  const int32_t* l1 = l0 + p.width;
  const int32_t n0 = checked_list(p, at0, nb, lane), n1 = two ? checked_list(p, at0 + 1, nb, lane) : 0;
  int32_t common = 0;
  if (n1 > 0)
    for (int32_t i0 = 0; i0 < n0; i0 += 32)
      common += __popc(__ballot_sync(0xffffffffu, i0 + lane < n0 && in_list(l1, n1, __ldg(l0 + min(i0 + lane, n0 - 1)))));
  int2* steps = p.steps + item * p.width;
  const uint32_t below = (1u << lane) - 1u;
  int32_t c = 0, r = common;
  for (int32_t i0 = 0; i0 < n0; i0 += 32) {
    const bool have = i0 + lane < n0;
    const int32_t v = __ldg(l0 + min(i0 + lane, n0 - 1));
    const bool both = have && n1 > 0 && in_list(l1, n1, v);
    const uint32_t mb = __ballot_sync(0xffffffffu, both), mh = __ballot_sync(0xffffffffu, have);
    if (both) steps[c + __popc(mb & below)] = make_int2(v, v);
    else if (have) steps[r + __popc(mh & ~mb & below)].x = v;
    c += __popc(mb);
    r += __popc(mh & ~mb);
  }
  r = common;
  for (int32_t i0 = 0; i0 < n1; i0 += 32) {
    const bool have = i0 + lane < n1;
    const int32_t v = __ldg(l1 + min(i0 + lane, n1 - 1));
    const bool alone = have && !(n0 > 0 && in_list(l0, n0, v));
    const uint32_t ma = __ballot_sync(0xffffffffu, alone);
    if (alone) steps[r + __popc(ma & below)].y = v;
    r += __popc(ma);
  }
  if (lane == 0) {
    // the step in which a tile meets the segment's last block, if that is a short one (the key mask)
    const bool ragged = (u.len & 127) != 0;
    const bool last0 = ragged && n0 > 0 && __ldg(l0 + n0 - 1) == nb - 1;
    const bool last1 = ragged && n1 > 0 && __ldg(l1 + n1 - 1) == nb - 1;
    d[0] = u.seg;
    d[1] = u.beg;
    d[2] = u.len;
    d[3] = h;
    d[4] = u.unit * 256;
    d[5] = n0;
    d[6] = n1;
    d[7] = common;
    d[8] = !last0 ? -1 : last1 ? common - 1 : n0 - 1;
    d[9] = !last1 ? -1 : last0 ? common - 1 : n1 - 1;
    d[10] = two ? 1 : 0;
    d[11] = 0;
    file_item(p, item, max(n0, n1));
  }
}

// Backward, first: one warp per (head, query block) marks itself at every key block of its list.
__global__ void __launch_bounds__(128) sparse_mark_kernel(const __grid_constant__ SparsePlanParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (blockIdx.x == 0) check_pack(p.cu, p.batch, p.total, p.max_seqlen, p.status, p.err_cu, p.err_max);
  write_maps(p, item, lane);
  if (item >= p.rows * p.heads) return;
  const int32_t h = static_cast<int32_t>(item / p.rows);
  const UnitAt u = unit_at(p.cu, p.batch, p.total, p.max_seqlen, item - h * p.rows, 7);
  if (!u.valid) return;
  const int32_t nb = (u.len + 127) >> 7;
  const int32_t n = checked_list(p, item, nb, lane);
  const int32_t* list = p.idx + item * p.width;
  const int64_t first = item - u.unit;  // row of the segment's first block, in this head
  for (int32_t i = lane; i < n; i += 32)
    atomicOr(p.bits + (first + __ldg(list + i)) * p.words + (u.unit >> 5), 1u << (u.unit & 31));
}

// Backward, second: one warp per (head, key block) counts the query blocks that name it.
__global__ void __launch_bounds__(128) sparse_plan_bwd_kernel(const __grid_constant__ SparsePlanParams p) {
  const int lane = threadIdx.x & 31;
  pdl_wait_primary();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (item >= p.rows * p.heads) return;
  const int32_t h = static_cast<int32_t>(item / p.rows);
  const UnitAt u = unit_at(p.cu, p.batch, p.total, p.max_seqlen, item - h * p.rows, 7);
  int32_t* d = p.desc + item * kDescInts;
  if (!u.valid) {
    if (lane == 0) p.cls[item] = -1;
    return;
  }
  int32_t n = 0;
  for (int32_t i = lane; i < p.words; i += 32) n += __popc(p.bits[item * p.words + i]);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    d[0] = u.seg;
    d[1] = u.beg;
    d[2] = u.len;
    d[3] = h;
    d[4] = u.unit * 128;
    d[5] = n;
    file_item(p, item, n);
  }
}

// The work order: the longest classes first (so that no long item is left for the end), and within a class the items
// as they lie, head by head.  The CTAs then work on one or two heads at a time, whose K and V stay in L2: with the
// items of a length in arbitrary order the forward of 16384 tokens, 24 heads took 516 us, as they lie 462 us.  Finer classes (2, 4 or 8
// an octave) change the forward by nothing and cost the backward of 65536 tokens 0 to 8 %.  Block c
// counts the items of longer classes and places those of class c.
constexpr int kOrderThreads = 1024;
__global__ void __launch_bounds__(kOrderThreads) sparse_order_kernel(const __grid_constant__ SparsePlanParams p) {
  __shared__ int32_t part[2][32];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int mine = blockIdx.x;
  const int64_t n = p.units * p.heads;
  const int4* cls = reinterpret_cast<const int4*>(p.cls);
  int32_t longer = 0, own = 0;
  for (int64_t i = threadIdx.x; i * 4 < n; i += kOrderThreads) {
    const int4 c = cls[i];
    const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool there = i * 4 + k < n;
      longer += there && v[k] > mine;
      own += there && v[k] == mine;
    }
  }
  longer = __reduce_add_sync(0xffffffffu, longer);
  own = __reduce_add_sync(0xffffffffu, own);
  if (lane == 0) {
    part[0][w] = longer;
    part[1][w] = own;
  }
  __syncthreads();
  int32_t base = 0, total = 0;
  for (int i = 0; i < 32; ++i) {
    base += part[0][i];
    total += part[1][i];
  }
  if (mine == 0 && threadIdx.x == 0) {
    p.counts[0] = base + total;
    p.counts[2] = 0;
  }
  if (total == 0) return;
  for (int64_t i0 = 0; i0 * 4 < n; i0 += kOrderThreads) {
    const int64_t i = i0 + threadIdx.x;
    const int4 c = i * 4 < n ? cls[i] : make_int4(-1, -1, -1, -1);
    const int v[4] = {c.x, c.y, c.z, c.w};
    int32_t have = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) have += i * 4 + k < n && v[k] == mine;
    int32_t x = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();  // the last turn's readers are done
    if (lane == 31) part[0][w] = x;
    __syncthreads();
    int32_t at = base + x - have;
    int32_t all = 0;
    for (int j = 0; j < 32; ++j) {
      if (j < w) at += part[0][j];
      all += part[0][j];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i * 4 + k < n && v[k] == mine) p.order[at++] = static_cast<int32_t>(i * 4 + k);
    base += all;
  }
}

}  // namespace pa
