// row_ring.h -- which row of a run goes through which stage of a ring in shared memory, and when its thread may start
// a copy.  How a copy is made and waited for is the caller's, so a host compiler takes this file too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define PA_RING_FN __device__ __forceinline__
#else
#define PA_RING_FN inline
#endif

namespace pa {

// The current row's stage, and the parity of its barrier's phase.
struct RingPlace {
  int stage = 0;
  uint32_t phase = 0;

  // those of the r-th row from the current one (r <= stages)
  PA_RING_FN bool wraps(int stages, int r) const { return r > 0 && stage + r >= stages; }
  PA_RING_FN int stage_of(int stages, int r) const { return wraps(stages, r) ? stage + r - stages : stage + r; }
  PA_RING_FN uint32_t phase_of(int stages, int r) const { return wraps(stages, r) ? phase ^ 1u : phase; }
  PA_RING_FN void advance(int stages, int n) {
    phase = phase_of(stages, n);
    stage = stage_of(stages, n);
  }
};

// The copies of a run's first rows (first, first + step, ... below end): load(stage, row) arms and starts one.
template <class Load>
PA_RING_FN void ring_start(int stages, int64_t first, int64_t step, int64_t end, Load load) {
  for (int s = 0; s < stages && first + s * step < end; ++s) load(s, first + s * step);
}

// The issuing thread, when the n rows from `row` on (in the stages from `at` on) have been worked on: their stages take
// the rows `stages` further on.  `landed` says that the copies of all n were seen to arrive.  If not (a wait gave up),
// a stage's barrier may be in the middle of a phase, so none is armed again, and drain(m) waits for the copies of the m
// rows in flight (the current one and those behind it): none must land in the memory of the block that comes after this
// one.  Returns false then: nothing more is to be started.
template <class Load, class Drain>
PA_RING_FN bool ring_refill(const RingPlace& at, int stages, int64_t row, int64_t step, int n, int64_t end, bool landed,
                            Load load, Drain drain) {
  if (__builtin_expect(!landed, 0)) {
    int m = 1;
    while (m < stages && row + m * step < end) ++m;
    drain(m);
    return false;
  }
  for (int r = 0; r < n && row + (r + stages) * step < end; ++r) load(at.stage_of(stages, r), row + (r + stages) * step);
  return true;
}

}  // namespace pa
