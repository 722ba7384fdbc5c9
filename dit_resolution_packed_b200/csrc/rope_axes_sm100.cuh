// rope_axes_sm100.cuh -- rotary positions with several axes on q and k [T, H, d], and the (cos, sin) table of a
// pack for the QKV projection's epilogue.
//
// Pair p of a head belongs to one axis a and turns by pos[t, a] * theta_a^(-2i/dims_a).  The kernel keeps angles
// in turns: t = pos * (frequency / 2 pi) and its distance to the nearest whole number in fp64, then sin and cos of
// that fraction in fp32, so a position of 2^24 loses nothing (the product's rounding is below 1e-9 turns).
//
// Bound by memory: q and k are read once and written once (4 tensors of 2 T H d bytes).  A block takes a few whole
// tokens, so the d/2 angles of a token are formed once for all its heads of q and k, while the block's first loads
// are in flight.
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace pa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 32;
constexpr int kRopeAhead = 3;  // units (of 32 bytes) that a thread has in flight, and about as many in all

// The pairs of a head: frequency in turns per position, and axis (fits the constant bank of a launch).
struct RopePairs {
  double turns[64];
  int8_t axis[64];  // -1: behind the axes, not rotated
  int32_t turned;   // pairs before those
};

struct RopeParams {
  const void* in[2];  // q, k (k may be missing: tensors = 1)
  void* out[2];
  const float* pos;  // [T, axes]
  int32_t total, heads, head_dim, axes, tensors, tokens;  // tokens per block
  float sign;             // -1: the inverse rotation
  float inv_per_token;    // 1 / units of a token
  RopePairs pairs;
};

// The launch's table of pairs as ordinary memory: its entries are read by lane (the constant bank would serve the 32
// lanes one after the other).
__device__ __forceinline__ const RopePairs* pairs_in_memory(const RopePairs& p) {
  const RopePairs* q;
  asm("mov.u64 %0, %1;" : "=l"(q) : "l"(&p));
  return q;
}

__device__ __forceinline__ float2 rope_cos_sin(const RopePairs* pairs, const float* pos, int axes, int64_t token,
                                               int pair, float sign) {
  const int a = pairs->axis[pair];
  if (a < 0) return make_float2(1.f, 0.f);
  const double t = static_cast<double>(pos[token * axes + a]) * pairs->turns[pair];
  const float f = static_cast<float>(2.0 * (t - rint(t)));
  float s, c;
  sincospif(f, &s, &c);
  return make_float2(c, sign * s);
}

// 8 pairs: (lo, hi) hold their first and second members (halves), or 16 neighbouring channels (interleaved).  kPart:
// only the first `turned` of them are rotated; the others keep their bits (a rotation by the angle 0 would not do: an
// infinity times 0 is NaN in its partner, and a -0 becomes 0).
template <bool kInter, bool kPart>
__device__ __forceinline__ void rope_unit(uint4& lo, uint4& hi, const float2* cs, int turned) {
  if (kPart && turned <= 0) return;
  float a[8], b[8];
  bf16x8_to_f32(lo, a);
  bf16x8_to_f32(hi, b);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 t = *reinterpret_cast<const float4*>(cs + i);  // (cos, sin) of pairs i and i + 1
    if (kInter) {
      float* x = i < 4 ? a + 2 * i : b + 2 * i - 8;
      const float x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3];
      x[0] = x0 * t.x - x1 * t.y;
      x[1] = x0 * t.y + x1 * t.x;
      x[2] = x2 * t.z - x3 * t.w;
      x[3] = x2 * t.w + x3 * t.z;
    } else {
      const float u0 = a[i], v0 = b[i], u1 = a[i + 1], v1 = b[i + 1];
      a[i] = u0 * t.x - v0 * t.y;
      b[i] = u0 * t.y + v0 * t.x;
      a[i + 1] = u1 * t.z - v1 * t.w;
      b[i + 1] = u1 * t.w + v1 * t.z;
    }
  }
  uint4 x = f32_to_bf16x8(a), y = f32_to_bf16x8(b);
  if (kPart && turned < 8) {
    // word w of a half holds a member each of pairs 2w and 2w + 1 (halves), or both members of a pair (interleaved)
    const auto keep = [&](uint32_t& to, uint32_t from, int pair) {
      const uint32_t mask = kInter ? (pair < turned ? 0u : ~0u)
                                   : (pair < turned ? 0u : 0xffffu) | (pair + 1 < turned ? 0u : 0xffff0000u);
      to = (to & ~mask) | (from & mask);
    };
    constexpr int step = kInter ? 1 : 2, second = kInter ? 4 : 0;
    keep(x.x, lo.x, 0);
    keep(x.y, lo.y, step);
    keep(x.z, lo.z, 2 * step);
    keep(x.w, lo.w, 3 * step);
    keep(y.x, hi.x, second);
    keep(y.y, hi.y, second + step);
    keep(y.z, hi.z, second + 2 * step);
    keep(y.w, hi.w, second + 3 * step);
  }
  lo = x;
  hi = y;
}

// kPart: the axes do not cover the head (with one kernel for both, heads that they cover took 2.5 % longer).
template <bool kInter, bool kPart>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float2 cs[kRopeMaxTokens * 64];
  const int half = p.head_dim >> 1;
  const int per_head = p.head_dim >> 4;             // units of a head
  const int per_tensor = p.heads * per_head;        // of a token in one tensor
  const int per_token = per_tensor * p.tensors;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.total - token0));
  const int units = tokens * per_token;
  // of a unit: its tensor, the element of its first 8 channels, the element distance to the other 8, its pairs
  auto locate = [&](int u, int& tensor, size_t& at, int& gap, int& pair0) {
    const int tok = static_cast<int>((static_cast<float>(u) + 0.5f) * p.inv_per_token);
    int rest = u - tok * per_token;
    tensor = rest >= per_tensor ? 1 : 0;
    rest -= tensor * per_tensor;
    const int sub = rest & (per_head - 1);
    at = (static_cast<size_t>(token0 + tok) * p.heads) * p.head_dim + static_cast<size_t>(rest - sub) * 16;
    at += kInter ? sub * 16 : sub * 8;
    gap = kInter ? 8 : half;
    pair0 = tok * half + sub * 8;
  };
  bool formed = false;
  for (int u0 = threadIdx.x; u0 < units || !formed; u0 += kRopeThreads * kRopeAhead) {
    uint4 lo[kRopeAhead], hi[kRopeAhead];
#pragma unroll
    for (int j = 0; j < kRopeAhead; ++j) {
      const int u = u0 + j * kRopeThreads;
      if (u < units) {
        int tensor, gap, pair0;
        size_t at;
        locate(u, tensor, at, gap, pair0);
        const uint16_t* src = static_cast<const uint16_t*>(p.in[tensor]) + at;
        lo[j] = *reinterpret_cast<const uint4*>(src);
        hi[j] = *reinterpret_cast<const uint4*>(src + gap);
      }
    }
    if (!formed) {  // every thread passes here once, in its first turn
      formed = true;
      for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads)
        cs[i] = rope_cos_sin(pairs_in_memory(p.pairs), p.pos, p.axes, token0 + i / half, i % half, p.sign);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kRopeAhead; ++j) {
      const int u = u0 + j * kRopeThreads;
      if (u < units) {
        int tensor, gap, pair0;
        size_t at;
        locate(u, tensor, at, gap, pair0);
        rope_unit<kInter, kPart>(lo[j], hi[j], cs + pair0, p.pairs.turned - (pair0 & (half - 1)));
        uint16_t* dst = static_cast<uint16_t*>(p.out[tensor]) + at;
        *reinterpret_cast<uint4*>(dst) = lo[j];
        *reinterpret_cast<uint4*>(dst + gap) = hi[j];
      }
    }
  }
}

struct RopeTableParams {
  const float* pos;
  float2* table;  // [T][d/2]
  int32_t total, half, axes;
  RopePairs pairs;
};

__global__ void __launch_bounds__(256) rope_axes_table_kernel(const __grid_constant__ RopeTableParams p) {
  pdl_launch_dependents();  // the projection reads the table in its epilogue only, behind its own wait
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t token = i / p.half;
  if (token >= p.total) return;
  p.table[i] = rope_cos_sin(pairs_in_memory(p.pairs), p.pos, p.axes, token, static_cast<int>(i - token * p.half), 1.f);
}

}  // namespace pa
