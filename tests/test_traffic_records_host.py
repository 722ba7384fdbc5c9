"""bench.py reports DRAM traffic only from records taken of the kernels as they are: the committed ones must match."""
import pytest

import bench


@pytest.mark.parametrize("record", ["attn_fwd_traffic.json", "attn_bwd_traffic.json"])
def test_the_committed_record_is_of_these_sources(record):
    rec = bench.traffic_for_current_kernel(record)
    assert rec is not None, f"profiles/{record}: the kernel's sources have changed since it was taken; take it again"
    assert rec["dram_bytes_per_launch"] == rec["dram_bytes_read_per_launch"] + rec["dram_bytes_write_per_launch"] > 0
