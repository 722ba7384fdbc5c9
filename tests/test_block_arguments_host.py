"""Arguments of the block operators that a call must not take at their word, on a machine without a GPU."""
import pytest
import torch

import dit_resolution_packed_b200 as pa
from dit_resolution_packed_b200 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return pa.load_library()


def _calls(ws):
    """Every call that takes scratch memory, with this one."""
    x = torch.zeros(300, 128, dtype=torch.bfloat16)
    q = x.view(300, 2, 64)
    cu = torch.tensor([0, 300], dtype=torch.int32)
    lse = torch.zeros(300, 2)
    idx, cnt = torch.zeros(2, 3, 2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    w = torch.ones(128, dtype=torch.bfloat16)
    yield lambda: pa.pa_block_norm_bwd(x, cu, None, None, x, x, None, None, None, None, None, torch.zeros(128), ws,
                                       pre="layer", w_pre=w)
    yield lambda: pa.pa_qkv_rope_axes_fwd(x, torch.zeros(384, 128, dtype=torch.bfloat16), torch.zeros(300, 1), [64],
                                          100.0, False, q, q, q, ws)
    yield lambda: pa.pa_block_select(q, q, cu, 300, 0.5, 1, idx, cnt, ws)
    yield lambda: pa.pa_block_sparse_attn_fwd(q, q, q, cu, 300, idx, cnt, 0.125, q, lse, ws)
    yield lambda: pa.pa_block_sparse_attn_bwd(q, q, q, q, lse, q, cu, 300, idx, cnt, 0.125, q, q, q, ws)


def test_a_workspace_has_the_bytes_that_it_names():
    """An expanded tensor's elements are one byte of memory: its count must not pass for a size."""
    one = torch.zeros(1, dtype=torch.uint8)
    for call in _calls(one.expand(1 << 30)):
        with pytest.raises(ValueError):
            call()
    for call in _calls(torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError):
            call()


def test_a_missing_or_small_workspace_is_refused():
    for ws in (None, torch.zeros(64, dtype=torch.uint8)):
        for call in _calls(ws):
            assert call() == pa.PA_ERR_WORKSPACE


def test_bytes_count_whatever_the_type():
    n = pa.pa_block_sparse_workspace_bytes(1, 300, 2, 64, 300, 2, 1)
    assert list(_calls(torch.zeros(n // 8 - 1, dtype=torch.int64)))[-1]() == pa.PA_ERR_WORKSPACE
    assert list(_calls(torch.zeros(n // 8 + 1, dtype=torch.int64)))[-1]() == pa.PA_ERR_NOT_DEVICE  # host memory


def test_a_list_table_too_wide_for_its_sizes_is_refused():
    """Bytes of the work lists grow with rows x width: past 63 bits the product must not pass for a small size."""
    lib = pa.load_library()
    wide, big = 2 ** 31 - 1, 2 ** 62
    for batch, total, heads, d in ((1 << 20, 1 << 23, 1 << 10, 64), (1, 2 ** 31 - 1, 100, 64)):
        for backward in (0, 1):
            assert pa.pa_block_sparse_workspace_bytes(batch, total, heads, d, total, wide, backward) == -1
        assert lib.pa_block_sparse_attn_fwd(16, 16, 16, 16, batch, total, heads, d, total, 16, 16, wide, 0.1, 16, 16, 16,
                                            big, None) == pa.PA_ERR_SHAPE
        assert lib.pa_block_sparse_attn_bwd(16, 16, 16, 16, 16, 16, 16, batch, total, heads, d, total, 16, 16, wide, 0.1,
                                            16, 16, 16, 16, big, None) == pa.PA_ERR_SHAPE
        assert lib.pa_block_select(16, 16, 16, batch, total, heads, d, 262144, 0.5, 1, wide, 16, 16, 16, big,
                                   None) == pa.PA_ERR_SHAPE
    # a table of 2^40 bytes is a size like any other
    assert pa.pa_block_sparse_workspace_bytes(1, 1 << 20, 8, 64, 1 << 20, 1 << 13, 0) > 0


def test_the_stride_of_a_single_row_is_nobodys():
    """With one image nothing steps from row to row, and the stride may be anything (1 in a tensor that came by DLPack)."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    row = torch.zeros(64, dtype=torch.bfloat16).as_strided((1, 64), (1, 1))
    z = torch.empty_like(x)
    assert pa.pa_block_norm_fwd(x, cu, None, None, z, pre="layer", scale=row, shift=row) == pa.PA_ERR_NOT_DEVICE


@pytest.mark.parametrize("density", [float("nan"), float("inf"), -float("inf"), -0.5, 1.5])
def test_a_density_that_is_none_is_refused_by_status(density):
    q = torch.zeros(300, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(pa.PackAttnError) as e:
        pa.block_select(q, q, torch.tensor([0, 300], dtype=torch.int32), 300, density)
    assert e.value.code == pa.PA_ERR_SCALE
