"""The entry points of packattn_block.h on a machine without a GPU: declared, exported, and refusing bad arguments
before any CUDA call."""
import ctypes
import math
import subprocess

import pytest
import torch

import dit_resolution_packed_b200 as pa
from dit_resolution_packed_b200 import _build, block


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def test_header_and_exports(lib):
    names = pa.header_functions(pa.BLOCK_HEADER_PATH)
    assert "pa_block_norm_fwd" in names and len(names) == len(set(names))
    out = subprocess.run(["nm", "-D", "--defined-only", pa.LIB_PATH], capture_output=True, text=True, check=True)
    exported = {line.split()[-1] for line in out.stdout.splitlines() if " T " in line}
    assert set(names) <= exported
    assert exported <= set(names) | set(pa.header_functions()) | {"_init", "_fini"}
    for name in names:
        assert getattr(lib, name).argtypes is not None, f"{name} has no declared argument types"


def test_status_strings():
    texts = [pa.status_string(c) for c in (pa.PA_ERR_WORKSPACE, pa.PA_ERR_BLOCKS, pa.PA_ERR_MODE)]
    assert len(set(texts)) == 3 and "unknown status" not in texts


# ---------------------------------------------------------------- norms

def _desc(**kw):
    base = dict(total_tokens=4, batch=1, hidden=64, residual_fp32=0, param_fp32=0, post=0, pre=1, residual_scale=1.0,
                eps=1e-6, cu_seqlens=4, gate=None, scale=None, shift=None, gate_stride=0, scale_stride=0,
                shift_stride=0, w_post=None, w_pre=None)
    base.update(kw)
    return block.BlockNormDesc(**base)


def _fwd(lib, x=16, y=None, r=None, z=16, **kw):
    return lib.pa_block_norm_fwd(ctypes.byref(_desc(**kw)), x, y, r, z, None)


def _bwd(lib, r=16, y=None, dr=16, dz=16, dx=16, dy=None, sums=(None,) * 5, ws=None, ws_bytes=0, **kw):
    return lib.pa_block_norm_bwd(ctypes.byref(_desc(**kw)), r, y, dr, dz, dx, dy, *sums, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(hidden=60), pa.PA_ERR_SHAPE), (dict(hidden=0), pa.PA_ERR_SHAPE), (dict(hidden=8200), pa.PA_ERR_SHAPE),
    (dict(total_tokens=-1), pa.PA_ERR_SHAPE), (dict(batch=-1), pa.PA_ERR_SHAPE), (dict(batch=0), pa.PA_ERR_SHAPE),
    (dict(eps=math.nan), pa.PA_ERR_SCALE), (dict(eps=-1.0), pa.PA_ERR_SCALE),
    (dict(y=16, r=16, residual_scale=math.inf), pa.PA_ERR_SCALE),
    (dict(pre=3), pa.PA_ERR_MODE), (dict(post=-1), pa.PA_ERR_MODE), (dict(residual_fp32=2), pa.PA_ERR_MODE),
    (dict(pre=0), pa.PA_ERR_MODE), (dict(z=None), pa.PA_ERR_MODE), (dict(pre=0, z=None), pa.PA_ERR_MODE),
    (dict(pre=0, z=None, y=16, r=16, scale=16), pa.PA_ERR_MODE),
    (dict(r=16), pa.PA_ERR_MODE), (dict(post=1), pa.PA_ERR_MODE), (dict(gate=16), pa.PA_ERR_MODE),
    (dict(residual_scale=0.5), pa.PA_ERR_MODE), (dict(w_post=16), pa.PA_ERR_MODE),
    (dict(x=None), pa.PA_ERR_NULL), (dict(y=16), pa.PA_ERR_NULL), (dict(scale=16, cu_seqlens=None), pa.PA_ERR_NULL),
    (dict(x=8), pa.PA_ERR_ALIGN), (dict(z=24), pa.PA_ERR_ALIGN), (dict(scale=24), pa.PA_ERR_ALIGN),
    (dict(scale=16, scale_stride=68), pa.PA_ERR_ALIGN), (dict(shift=16, shift_stride=-64), pa.PA_ERR_SHAPE),
    (dict(w_pre=4), pa.PA_ERR_ALIGN), (dict(scale=16, cu_seqlens=6), pa.PA_ERR_ALIGN),
    (dict(total_tokens=0), pa.PA_OK), (dict(total_tokens=0, batch=0), pa.PA_OK),
])
def test_norm_fwd_refusals(lib, kw, code):
    assert _fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dz=None), pa.PA_ERR_MODE), (dict(pre=0), pa.PA_ERR_MODE), (dict(pre=0, dz=None, dr=None), pa.PA_ERR_MODE),
    (dict(y=16), pa.PA_ERR_MODE), (dict(dy=16), pa.PA_ERR_MODE), (dict(r=None), pa.PA_ERR_NULL),
    (dict(pre=0, dz=None), pa.PA_ERR_MODE),
    (dict(dx=None), pa.PA_ERR_NULL), (dict(dx=20), pa.PA_ERR_ALIGN),
    (dict(sums=(16, None, None, None, None)), pa.PA_ERR_MODE),
    (dict(sums=(None, None, None, None, 16)), pa.PA_ERR_MODE),
    (dict(sums=(None, 16, None, None, None), scale=16), pa.PA_ERR_WORKSPACE),
    (dict(sums=(None, 16, None, None, None), scale=16, ws=16, ws_bytes=64), pa.PA_ERR_WORKSPACE),
    (dict(sums=(None, 16, None, None, None), scale=16, ws=8, ws_bytes=1 << 20), pa.PA_ERR_WORKSPACE),
    (dict(sums=(None, 24, None, None, None), scale=16, ws=16, ws_bytes=1 << 20), pa.PA_ERR_ALIGN),
    (dict(total_tokens=0), pa.PA_OK),
])
def test_norm_bwd_refusals(lib, kw, code):
    assert _bwd(lib, **kw) == code


def test_norm_null_desc_and_workspace(lib):
    assert lib.pa_block_norm_fwd(None, 16, None, None, 16, None) == pa.PA_ERR_NULL
    assert lib.pa_block_norm_bwd(None, *([16] * 11), 16, 0, None) == pa.PA_ERR_NULL
    assert pa.pa_block_norm_workspace_bytes(-1, 4, 64) == -1
    assert pa.pa_block_norm_workspace_bytes(1, 4, 65) == -1
    # per image three rows of channels for each of 8 teams, and two more
    assert pa.pa_block_norm_workspace_bytes(2, 0, 64) == 4 * (2 * 8 * 3 + 2 * 2) * 64
    # runs of rows, not rows: bounded however long the pack is
    assert 0 < pa.pa_block_norm_workspace_bytes(1, 2 ** 31 - 1, 8192) < 2 ** 28
    assert pa.pa_block_norm_workspace_bytes(2 ** 20, 2 ** 31 - 1, 8192) > 2 ** 35


def test_norm_python_checks():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    m = torch.zeros(1, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pa.block_norm_fwd(x.half(), cu)
    with pytest.raises(TypeError):
        pa.block_norm_fwd(x, cu, scale=m, shift=m.float())
    with pytest.raises(TypeError):
        pa.block_norm_fwd(x, cu.long(), scale=m)
    with pytest.raises(ValueError):
        pa.block_norm_fwd(x, None, scale=m)
    with pytest.raises(ValueError):
        pa.block_norm_fwd(x, cu, pre="batch")
    with pytest.raises(ValueError):
        pa.block_norm_fwd(x, cu, scale=m[:, :32])
    with pytest.raises(ValueError):
        pa.block_norm_fwd(torch.zeros(64, 4, dtype=torch.bfloat16).t(), cu)
    with pytest.raises(ValueError):
        pa.block_norm_fwd(x, cu, w_pre=m)
    with pytest.raises(pa.PackAttnError) as e:
        pa.block_norm_fwd(x, cu, residual_scale=0.5)
    assert e.value.code == pa.PA_ERR_MODE


# ---------------------------------------------------------------- rotary positions with several axes

def _axes(dims=(32, 32), theta=(100.0, 100.0), inter=0, axes=None):
    d = block.RopeAxesDesc(axes=len(dims) if axes is None else axes, interleaved=inter)
    for i, (n, b) in enumerate(zip(dims, theta)):
        d.dims[i], d.theta[i] = n, b
    return ctypes.byref(d)


def _rope(lib, q=16, k=16, pos=16, total=4, heads=2, d=64, desc=None, inverse=0, qo=16, ko=16):
    return lib.pa_rope_axes(q, k, pos, total, heads, d, _axes() if desc is None else desc, inverse, qo, ko, None)


def _qkv(lib, x=16, w=16, pos=16, total=4, hidden=64, heads=2, d=64, desc=None, q=16, k=16, v=16, ws=16,
         ws_bytes=1 << 20):
    return lib.pa_qkv_rope_axes_fwd(x, w, pos, total, hidden, heads, d, _axes() if desc is None else desc, q, k, v, ws,
                                    ws_bytes, None)


def test_rope_refusals(lib):
    for call in (_rope, _qkv):
        assert call(lib, d=96) == pa.PA_ERR_HEAD_DIM
        assert call(lib, heads=0) == pa.PA_ERR_SHAPE
        assert call(lib, total=-1) == pa.PA_ERR_SHAPE
        assert call(lib, total=0) == pa.PA_OK
        assert call(lib, desc=_axes(dims=(31, 32))) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(dims=(0, 32))) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(dims=(-2, 32))) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(dims=(34, 32))) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(axes=0)) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(axes=5)) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(inter=2)) == pa.PA_ERR_SHAPE
        assert call(lib, desc=_axes(theta=(0.0, 1.0))) == pa.PA_ERR_SCALE
        assert call(lib, desc=_axes(theta=(math.inf, 1.0))) == pa.PA_ERR_SCALE
        assert call(lib, pos=None) == pa.PA_ERR_NULL
        assert call(lib, pos=18) == pa.PA_ERR_ALIGN
        assert call(lib, q=8) == pa.PA_ERR_ALIGN
        assert call(lib, k=None) == pa.PA_ERR_NULL
    assert lib.pa_rope_axes(16, 16, 16, 4, 2, 64, None, 0, 16, 16, None) == pa.PA_ERR_NULL
    assert _rope(lib, inverse=2) == pa.PA_ERR_SHAPE
    assert _rope(lib, qo=None) == pa.PA_ERR_NULL
    assert _rope(lib, heads=1 << 20) == pa.PA_ERR_SHAPE
    assert _qkv(lib, hidden=12) == pa.PA_ERR_SHAPE
    assert _qkv(lib, ws=None) == pa.PA_ERR_WORKSPACE
    assert _qkv(lib, ws_bytes=4 * 32 * 8 - 1) == pa.PA_ERR_WORKSPACE
    assert pa.pa_rope_axes_workspace_bytes(4, 64) == 4 * 32 * 8
    assert pa.pa_rope_axes_workspace_bytes(-1, 64) == -1 and pa.pa_rope_axes_workspace_bytes(4, 80) == -1
    q, pos = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        pa.rope_axes_fwd(q, q, pos, [16, 16, 16])
    with pytest.raises(ValueError):
        pa.rope_axes_fwd(q, q, pos, [32, 32], [1.0])
    with pytest.raises(ValueError):
        pa.rope_axes_fwd(q, q, pos[:3], [32, 32])
    with pytest.raises(TypeError):
        pa.rope_axes_fwd(q, q, pos.double(), [32, 32])
    with pytest.raises(TypeError):
        pa.rope_axes_fwd(q, q.float(), pos, [32, 32])


# ---------------------------------------------------------------- attention over selected blocks

BIG = 1 << 40


def _select(lib, q=16, k=16, cu=16, batch=1, total=300, heads=2, d=64, longest=300, density=0.5, floor=1, width=2, idx=16,
            cnt=16, ws=16, ws_bytes=BIG):
    return lib.pa_block_select(q, k, cu, batch, total, heads, d, longest, density, floor, width, idx, cnt, ws, ws_bytes,
                               None)


def _sfwd(lib, q=16, k=16, v=16, cu=16, batch=1, total=300, heads=2, d=64, longest=300, idx=16, cnt=16, width=2,
          scale=0.125, out=16, lse=16, ws=16, ws_bytes=BIG):
    return lib.pa_block_sparse_attn_fwd(q, k, v, cu, batch, total, heads, d, longest, idx, cnt, width, scale, out, lse, ws,
                                        ws_bytes, None)


def _sbwd(lib, q=16, k=16, v=16, out=16, lse=16, dout=16, cu=16, batch=1, total=300, heads=2, d=64, longest=300, idx=16,
          cnt=16, width=2, scale=0.125, dq=16, dk=16, dv=16, ws=16, ws_bytes=BIG):
    return lib.pa_block_sparse_attn_bwd(q, k, v, out, lse, dout, cu, batch, total, heads, d, longest, idx, cnt, width,
                                        scale, dq, dk, dv, ws, ws_bytes, None)


def test_sparse_refusals(lib):
    for call in (_select, _sfwd, _sbwd):
        assert call(lib, d=96) == pa.PA_ERR_HEAD_DIM
        assert call(lib, heads=0) == pa.PA_ERR_SHAPE
        assert call(lib, heads=1 << 20) == pa.PA_ERR_SHAPE
        assert call(lib, batch=-1) == pa.PA_ERR_SHAPE
        assert call(lib, batch=0) == pa.PA_ERR_SHAPE
        assert call(lib, total=-1) == pa.PA_ERR_SHAPE
        assert call(lib, width=0) == pa.PA_ERR_SHAPE
        assert call(lib, batch=0, total=0) == pa.PA_OK
        assert call(lib, longest=0) == pa.PA_ERR_MAX_SEQLEN
        for name in ("q", "k", "cu", "idx", "cnt"):
            assert call(lib, **{name: None}) == pa.PA_ERR_NULL, name
            assert call(lib, **{name: 18}) == pa.PA_ERR_ALIGN, name
        assert call(lib, ws=None) == pa.PA_ERR_WORKSPACE
        assert call(lib, ws=24) == pa.PA_ERR_WORKSPACE
        assert call(lib, ws_bytes=1000) == pa.PA_ERR_WORKSPACE
    assert _select(lib, density=-0.1) == pa.PA_ERR_SCALE and _select(lib, density=1.5) == pa.PA_ERR_SCALE
    assert _select(lib, density=math.nan) == pa.PA_ERR_SCALE
    assert _select(lib, floor=0) == pa.PA_ERR_SHAPE
    assert _select(lib, width=1) == pa.PA_ERR_BLOCKS  # ceil(0.5 * 3) = 2 blocks
    assert _select(lib, total=1 << 20, longest=262145) == pa.PA_ERR_MAX_SEQLEN
    for call in (_sfwd, _sbwd):
        assert call(lib, total=0) == pa.PA_OK
        assert call(lib, scale=math.inf) == pa.PA_ERR_SCALE
        for name in ("v", "out", "lse"):
            assert call(lib, **{name: None}) == pa.PA_ERR_NULL, name
        assert call(lib, v=8) == pa.PA_ERR_ALIGN and call(lib, lse=2) == pa.PA_ERR_ALIGN
    for name in ("dout", "dq", "dk", "dv"):
        assert _sbwd(lib, **{name: None}) == pa.PA_ERR_NULL
        assert _sbwd(lib, **{name: 8}) == pa.PA_ERR_ALIGN


def test_sparse_sizes(lib):
    assert pa.pa_block_rows(3, 1000) == 10 and pa.pa_block_rows(-1, 5) == -1 and pa.pa_block_rows(1, -5) == -1
    assert pa.pa_block_select_workspace_bytes(3, 1000, 2, 64) == 2 * 8 * 10 * 2 * 64
    assert pa.pa_block_select_workspace_bytes(3, 1000, 2, 65) == -1
    assert pa.pa_block_sparse_workspace_bytes(1, 300, 2, 65, 300, 2, 0) == -1
    assert pa.pa_block_sparse_workspace_bytes(1, 300, 2, 64, -1, 2, 0) == -1
    fwd, bwd = (pa.pa_block_sparse_workspace_bytes(1, 65536, 8, 64, 65536, 32, b) for b in (0, 1))
    assert fwd > 8 * 256 * 32 * 8 and bwd > 65536 * 8 * 64 * 4
    # an 8M-token pack: sizes past 32 bits
    assert pa.pa_block_sparse_workspace_bytes(1, 1 << 23, 8, 128, 1 << 23, 64, 1) > 1 << 33


def test_sparse_python_checks():
    q = torch.zeros(300, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 300], dtype=torch.int32)
    idx, cnt = torch.zeros(2, 3, 2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.block_sparse_attn_fwd(q, q, q, cu, 300, idx[:, :2], cnt)
    with pytest.raises(TypeError):
        pa.block_sparse_attn_fwd(q, q, q, cu, 300, idx.long(), cnt)
    with pytest.raises(ValueError):
        pa.block_sparse_attn_fwd(q, q[:200], q, cu, 300, idx, cnt)
    with pytest.raises(ValueError):
        pa.block_sparse_attn_bwd(q, q, q, q, torch.zeros(2, 300), q, cu, 300, idx, cnt)
    with pytest.raises(TypeError):
        pa.block_select(q.float(), q, cu, 300, 0.5)
    with pytest.raises(pa.PackAttnError):
        pa.block_select(q, q, cu, 300, 2.0)
