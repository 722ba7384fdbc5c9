"""The kernels' sources, read: a warp hands an item's slot back to the producer only when all its lanes have read it.

One lane arrives for the warp.  Unless the warp comes together between the reads and that arrival (a __syncwarp, or a vote
on what was read), another lane may still be reading when the producer writes the next item there.
"""
import os
import re

from dit_resolution_packed_b200 import _build

READ = re.compile(r"\b(?:next_item_from_ring|bwd_next_item|sparse_next)\(bars, sk")


def test_every_release_stands_behind_the_whole_warps_reads():
    seen = 0
    for name in _build.HEADERS:
        with open(os.path.join(_build.CSRC, name)) as f:
            src = re.sub(r"//[^\n]*", "", f.read())
        for m in READ.finditer(src):
            end = src.index("mbar_arrive(&bars->sched_empty[", m.end())
            assert "__syncwarp()" in src[m.end():end] or "__any_sync(0xffffffffu, got <= 0)" in src[m.end():end], f"{name}:{src.count(chr(10), 0, m.start()) + 1}"
            seen += 1
    assert seen == 9  # the MMA and math warps of four kernels (the backward has two kinds of math warps)
