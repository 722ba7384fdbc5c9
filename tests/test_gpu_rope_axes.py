"""Rotary positions with several axes (pa_rope_axes, pa_qkv_rope_axes_fwd) on the GPU vs the fp64 oracle.

Tolerances: an output is rounded to bf16 once (half a step, 2^-8 of its value).  Before it, cos and sin are fp32 of
an angle reduced in fp64 (within 4 x 2^-24 each) and each output is two products and a sum: 8 x 2^-24 of |a| + |b|.
The projection sums C products in fp32 (C + 8 roundings of the sum of their magnitudes at most).
"""
import numpy as np
import pytest
import torch

import dit_resolution_packed_b200 as pa
from oracle import block as ob

pytestmark = pytest.mark.gpu
HALF, EPS32 = 2.0 ** -8, 2.0 ** -24


def _inputs(T, H, d, axes, seed, far=64.0, whole=True):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(T, H, d, generator=g).to(torch.bfloat16) for _ in range(2))
    pos = torch.rand(T, axes, generator=g) * far
    return q, k, torch.floor(pos) if whole else pos


def _check(got, x, pos, dims, theta, inter, inverse, what):
    ref = ob.rope_axes(x, pos, dims, theta, inter, inverse)
    mag = np.abs(ob.f64(x)).max(-1, keepdims=True) * 2
    err = np.abs(got.double().cpu().numpy() - ref)
    bound = np.abs(ref) * HALF * (1 + HALF) + 8 * EPS32 * mag
    assert (err <= bound).all(), f"{what}: worst {float((err / bound).max()):.2f} of the bound"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,dims", [(64, [64]), (64, [16, 24, 24]), (64, [8, 16]), (64, [2, 2, 2, 58]),
                                    (128, [16, 56, 56]), (128, [32, 32, 32, 32]), (128, [128]), (128, [6, 50])])
@pytest.mark.parametrize("T,H", [(1, 1), (7, 3), (1000, 5), (37, 24)])
def test_matches_fp64(cuda_device, T, H, d, dims, inter):
    q, k, pos = _inputs(T, H, d, len(dims), 1)
    for fn, inverse in ((pa.rope_axes_fwd, False), (pa.rope_axes_bwd, True)):
        a, b = fn(q.to(cuda_device), k.to(cuda_device), pos.to(cuda_device), dims, 100.0, inter)
        assert pa.pa_get_error() == pa.PA_OK
        _check(a, q, pos, dims, 100.0, inter, inverse, "q")
        _check(b, k, pos, dims, 100.0, inter, inverse, "k")


def test_far_and_fractional_positions(cuda_device):
    dims, theta = [32, 16, 16], [10000.0, 30.0, 2.0]
    for far, whole in ((2.0 ** 24, True), (3.0, False)):
        q, k, pos = _inputs(130, 2, 64, 3, 2, far, whole)
        pos[0] = -pos[0]
        a, b = pa.rope_axes_fwd(q.to(cuda_device), k.to(cuda_device), pos.to(cuda_device), dims, theta)
        _check(a, q, pos, dims, theta, False, False, "q")
        _check(b, k, pos, dims, theta, False, False, "k")


def test_channels_behind_the_axes_are_copied(cuda_device):
    q, k, pos = _inputs(50, 3, 128, 1, 3)
    a, b = pa.rope_axes_fwd(q.to(cuda_device), k.to(cuda_device), pos.to(cuda_device), [32])
    for got, x in ((a, q), (b, k)):
        assert torch.equal(got.cpu()[..., 16:64], x[..., 16:64]) and torch.equal(got.cpu()[..., 80:], x[..., 80:])


def test_q_alone_in_place_and_no_tokens(cuda_device):
    q, k, pos = _inputs(300, 4, 64, 2, 4)
    dims = [32, 32]
    a, b = pa.rope_axes_fwd(q.to(cuda_device), k.to(cuda_device), pos.to(cuda_device), dims)
    alone, none = pa.rope_axes_fwd(q.to(cuda_device), None, pos.to(cuda_device), dims)
    assert none is None and torch.equal(alone, a)
    q2, k2 = q.to(cuda_device), k.to(cuda_device)
    assert pa.pa_rope_axes(q2, k2, pos.to(cuda_device), dims, 10000.0, False, False, q2, k2) == pa.PA_OK
    assert torch.equal(q2, a) and torch.equal(k2, b)
    e, _ = pa.rope_axes_fwd(q2[:0], k2[:0], pos.to(cuda_device)[:0], dims)
    assert e.shape[0] == 0


def test_a_nan_position_stays_in_its_token(cuda_device):
    q, k, pos = _inputs(20, 2, 64, 2, 5)
    want, _ = pa.rope_axes_fwd(q.to(cuda_device), k.to(cuda_device), pos.to(cuda_device), [32, 32])
    pos[3, 1] = float("inf")
    got, _ = pa.rope_axes_fwd(q.to(cuda_device), k.to(cuda_device), pos.to(cuda_device), [32, 32])
    keep = torch.arange(20) != 3
    assert torch.equal(got.cpu()[keep], want.cpu()[keep]) and torch.isnan(got[3, :, 16:32].float()).all()
    assert torch.equal(got[3, :, :16], want[3, :, :16])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,C,H,d,dims", [(1, 64, 1, 64, [64]), (300, 192, 5, 64, [8, 24, 24]),
                                          (517, 136, 3, 128, [16, 56, 56]), (129, 520, 2, 128, [32, 32])])
def test_projection(cuda_device, T, C, H, d, dims, inter):
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, C, generator=g).to(torch.bfloat16)
    w = (torch.randn(3 * H * d, C, generator=g) * C ** -0.5).to(torch.bfloat16)
    pos = torch.floor(torch.rand(T, len(dims), generator=g) * 100)
    q, k, v = pa.qkv_rope_axes_fwd(x.to(cuda_device), w.to(cuda_device), pos.to(cuda_device), H, d, dims, 100.0, inter)
    assert pa.pa_get_error() == pa.PA_OK
    y = (ob.f64(x) @ ob.f64(w).T).reshape(T, 3, H, d)
    mag = (np.abs(ob.f64(x)) @ np.abs(ob.f64(w)).T).reshape(T, 3, H, d)
    for i, (got, name) in enumerate(((q, "q"), (k, "k"), (v, "v"))):
        ref = ob.rope_axes(y[:, i], pos, dims, 100.0, inter) if i < 2 else y[:, i]
        err = np.abs(got.double().cpu().numpy() - ref)
        bound = np.abs(ref) * HALF * (1 + HALF) + 2 * (C + 16) * EPS32 * mag[:, i].max(-1, keepdims=True)
        assert (err <= bound).all(), f"{name}: worst {float((err / bound).max()):.2f}"


def test_projection_with_one_axis_is_the_existing_one(cuda_device):
    """One axis over all channels, positions restarting at every image: pa_qkv_rope_fwd, to an ulp of its table."""
    lens, H, d, C = [40, 3, 90], 2, 64, 128
    g = torch.Generator().manual_seed(7)
    x = torch.randn(sum(lens), C, generator=g).to(torch.bfloat16).to(cuda_device)
    w = (torch.randn(3 * H * d, C, generator=g) * C ** -0.5).to(torch.bfloat16).to(cuda_device)
    cu = torch.tensor([0, 40, 43, 133], dtype=torch.int32, device=cuda_device)
    pos = torch.cat([torch.arange(n) for n in lens]).float()[:, None].to(cuda_device)
    a = pa.qkv_rope_fwd(x, w, cu, 90, H, d)
    b = pa.qkv_rope_axes_fwd(x, w, pos, H, d, [d])
    assert torch.equal(a[2], b[2])
    for s, t in zip(a[:2], b[:2]):
        assert torch.allclose(s.float(), t.float(), rtol=2.0 ** -7, atol=1e-5)


def test_streams_and_graphs(cuda_device):
    q, k, pos = (t.to(cuda_device) for t in _inputs(900, 6, 64, 3, 8))
    x = torch.randn(900, 128, device=cuda_device).to(torch.bfloat16)
    w = (torch.randn(3 * 6 * 64, 128, device=cuda_device) * 0.1).to(torch.bfloat16)
    dims = [16, 24, 24]

    def both(stream=None):
        return pa.rope_axes_fwd(q, k, pos, dims, stream=stream) + pa.qkv_rope_axes_fwd(x, w, pos, 6, 64, dims,
                                                                                      stream=stream)
    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(side)
    assert pa.pa_get_error(side) == pa.PA_OK and all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
