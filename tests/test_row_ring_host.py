"""The ring of rows of the norm kernels (``csrc/row_ring.h``), compiled for the host and run against model barriers.

A copy that does not come within the limit makes a wait give up.  From then on no barrier may be armed while its phase is
open, and no copy may be in flight when the block ends.
"""
import os
import subprocess

import pytest

from dit_resolution_packed_b200 import _build

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "row_ring.h"

// A barrier per stage: `done` phases completed, and whether the current one is armed (a copy in flight).
struct Bar { unsigned done = 0; bool armed = false; int64_t row = -1; };

struct Model {
  std::vector<Bar> bars;
  int64_t late;  // this row's copy comes only to those who drain; those behind it may come or not
  bool gave_up = false;
  int faults = 0;
  unsigned seed;
  bool chance() { seed = seed * 1664525u + 1013904223u; return seed >> 31; }
  void load(int s, int64_t row) {
    if (bars[s].armed) ++faults;  // armed again in the middle of a phase
    bars[s].armed = true;
    bars[s].row = row;
  }
  void land(int s) { bars[s].armed = false; ++bars[s].done; }
  bool wait(int s, uint32_t parity, int64_t row) {
    Bar& b = bars[s];
    if (b.armed && b.row == row && row != late && !(row > late && late >= 0 && chance())) land(s);
    const bool ok = (b.done & 1u) != parity;
    if (!ok) gave_up = true;
    return ok;
  }
  void drain(int s, uint32_t parity) {
    if (bars[s].armed ? (bars[s].done & 1u) != parity : (bars[s].done & 1u) == parity) ++faults;  // the wrong phase
    if (bars[s].armed) land(s);
  }
};

// vote: the issuing thread hears of every wait (as in the kernels); else it goes on whatever the waits said.
int run(int stages, int tile, int64_t rows, int64_t step, int64_t late, bool vote, unsigned seed) {
  Model m;
  m.bars.resize(stages);
  m.late = late;
  m.seed = seed;
  auto load = [&](int s, int64_t r) { m.load(s, r); };
  pa::RingPlace at;
  auto drain = [&](int rows) {
    for (int r = 0; r < rows; ++r) m.drain(at.stage_of(stages, r), at.phase_of(stages, r));
  };
  const int64_t end = rows * step;
  pa::ring_start(stages, 0, step, end, load);
  bool issuing = true;
  for (int64_t row = 0; row < end;) {
    int n = 0;
    bool landed = true;
    for (; n < tile && row + n * step < end; ++n)
      landed = m.wait(at.stage_of(stages, n), at.phase_of(stages, n), row + n * step) && landed;
    if (issuing) issuing = pa::ring_refill(at, stages, row, step, n, end, landed || !vote, load, drain);
    at.advance(stages, n);
    row += n * step;
  }
  for (auto& b : m.bars) m.faults += b.armed;  // in flight at the end
  if (m.gave_up != (late >= 0)) ++m.faults;
  return m.faults;
}

int main(int argc, char** argv) {
  const bool vote = std::atoi(argv[1]) != 0;
  long runs = 0, bad = 0;
  for (int stages = 1; stages <= 9; ++stages)
    for (int tile = 1; tile <= stages; ++tile)
      for (int64_t rows : {1, 2, 5, 8, 17, 40})
        for (int64_t step : {1, 3})
          for (int64_t late = -1; late < rows; ++late)
            for (unsigned seed = 1; seed <= 3; ++seed, ++runs)
              bad += run(stages, tile, rows, step, late < 0 ? -1 : late * step, vote, seed * 77u + late) != 0;
  std::printf("%ld %ld\n", runs, bad);
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, exe = d / "model.cc", d / "model"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, str(src), "-o", str(exe)], check=True)
    return lambda vote: [int(x) for x in subprocess.run([str(exe), str(vote)], capture_output=True, text=True,
                                                        check=True).stdout.split()]


def test_a_wait_that_gives_up_ends_the_copies(model):
    runs, bad = model(1)
    assert runs > 10000 and bad == 0


def test_the_model_sees_a_refill_that_does_not_ask(model):
    """An issuing thread that ignores what the waits said arms open barriers or leaves copies in flight."""
    runs, bad = model(0)
    assert bad > runs // 2


def test_the_kernels_use_it():
    with open(os.path.join(_build.CSRC, "block_norm_sm100.cuh")) as f:
        src = f.read()
    assert src.count("ring_refill(") == 2 and src.count("ring_start(") == 2
    # every wait goes through the ring, and what it said (through the block's flag) is asked before a refill
    assert src.count("mbar_wait(") == 1 and src.count("const bool landed = *wc.abort_flag == 0;") == 2
