"""The operators of a DiT block run together, as a model runs them: norm -> QKV + rotary positions -> selection of key
blocks -> sparse attention -> output projection -> gated residual join with the next norm, and back.  Each stage is
held against the fp64 oracle on its own inputs (the GPU's outputs of the stage before), and the whole chain's gradient
against differences of the fp64 chain."""
import numpy as np
import pytest
import torch

import dit_resolution_packed_b200 as pa
import workloads
from oracle import block as ob
from oracle import proj
from tests import parity

pytestmark = pytest.mark.gpu

LENS, C, H, D = [300, 129, 0, 560], 256, 2, 128
DIMS, THETA = [16, 56, 56], 1000.0


def _rn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def _model(seed):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(LENS), len(LENS)
    mod = _rn(g, B, 6, C, scale=0.3)
    pos = torch.cat([torch.stack([torch.zeros(n), torch.arange(n) // 20, torch.arange(n) % 20], 1) for n in LENS]).float()
    return dict(x=_rn(g, T, C), mod=mod, w_qkv=_rn(g, 3 * H * D, C, scale=C ** -0.5), w_o=_rn(g, C, H * D, scale=0.1),
                w_post=_rn(g, C, scale=0.2) + 1, pos=pos, cu=workloads.cu_seqlens_from_lengths(LENS),
                dr=_rn(g, T, C), dz=_rn(g, T, C))


def _forward(m, stream=None):
    """One block, every stage's output by name."""
    s = dict(stream=stream)
    longest, cu, mod = max(LENS), m["cu"], m["mod"]
    _, h = pa.block_norm_fwd(m["x"], cu, pre="layer", scale=mod[:, 1], shift=mod[:, 0], **s)
    q, k, v = pa.qkv_rope_axes_fwd(h, m["w_qkv"], m["pos"], H, D, DIMS, THETA, **s)
    idx, cnt = pa.block_select(q, k, cu, longest, 0.5, 2, **s)
    o, lse = pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt, **s)
    y = pa.linear_fwd(o.view(o.shape[0], -1), m["w_o"], **s)
    r, z = pa.block_norm_fwd(m["x"], cu, y=y, gate=mod[:, 2], post="rms", w_post=m["w_post"], pre="layer",
                             scale=mod[:, 4], shift=mod[:, 3], **s)
    return dict(h=h, q=q, k=k, v=v, idx=idx, cnt=cnt, o=o, lse=lse, y=y, r=r, z=z)


def _backward(m, f, stream=None):
    """Gradients of the block's q, k (before the rotation), v, y and modulation from dr and dz."""
    s = dict(stream=stream)
    cu, mod, longest = m["cu"], m["mod"], max(LENS)
    join = pa.block_norm_bwd(f["r"], cu, m["dr"], m["dz"], y=f["y"], gate=mod[:, 2], post="rms", w_post=m["w_post"],
                             pre="layer", scale=mod[:, 4], shift=mod[:, 3], **s)
    do = pa.linear_fwd(join["dy"], m["w_o"].t().contiguous(), **s).view(f["o"].shape)
    dq, dk, dv = pa.block_sparse_attn_bwd(f["q"], f["k"], f["v"], f["o"], f["lse"], do, cu, longest, f["idx"], f["cnt"],
                                          **s)
    dqr, dkr = pa.rope_axes_bwd(dq, dk, m["pos"], DIMS, THETA, **s)
    w = m["w_qkv"].view(3, -1, C)
    dh = sum(pa.linear_fwd(d.reshape(d.shape[0], -1), w[i].t().contiguous(), **s).float()
             for i, d in enumerate((dqr, dkr, dv))).to(torch.bfloat16)
    front = pa.block_norm_bwd(m["x"], cu, None, dh, pre="layer", scale=mod[:, 1], shift=mod[:, 0], **s)
    return dict(join=join, do=do, dq=dq, dk=dk, dv=dv, dqr=dqr, dkr=dkr, dh=dh, front=front,
                dx=join["dx"].float() + front["dx"].float())


def _gpu(m, dev):
    return {k: v.to(dev) for k, v in m.items()}


def _f(t):
    return t.double().cpu().numpy()


def test_block_stage_by_stage(cuda_device):
    m = _model(1)
    f = _forward(_gpu(m, cuda_device))
    b = _backward(_gpu(m, cuda_device), f)
    assert pa.pa_get_error() == pa.PA_OK
    cu, mod = m["cu"].numpy(), m["mod"]

    def near(got, ref, rel, what):
        err = np.linalg.norm(_f(got) - ref) / max(np.linalg.norm(ref), 1e-30)
        assert err <= rel, f"{what}: {err}"

    # rounding to bf16 alone is 2^-8 / sqrt(3) of a value at most; products of rounded factors a few times that
    near(f["h"], ob.front(m["x"], cu, "layer", None, mod[:, 1], mod[:, 0]), 3e-3, "h")
    rq, rk, rv = proj.qkv_rope(f["h"].cpu(), m["w_qkv"], cu, H, D, 0.0)
    near(f["v"], rv, 3e-3, "v")
    near(f["q"], ob.rope_axes(rq, m["pos"], DIMS, THETA), 3e-3, "q")
    near(f["k"], ob.rope_axes(rk, m["pos"], DIMS, THETA), 3e-3, "k")
    ri, rc = ob.block_select(f["q"], f["k"], cu, 0.5, 2, f["idx"].shape[2])
    assert np.array_equal(ri, f["idx"].cpu().numpy()) and np.array_equal(rc, f["cnt"].cpu().numpy())
    ro, rl = ob.sparse_attention(f["q"], f["k"], f["v"], cu, ri, rc, D ** -0.5)
    near(f["o"], ro, 4e-3, "o")
    assert np.abs(_f(f["lse"]) - rl).max() <= 2e-4
    parity.proj_check(_f(f["y"]), proj.linear(f["o"].view(-1, H * D).cpu(), m["w_o"]), "y")
    near(f["r"], ob.join(m["x"], cu, f["y"], mod[:, 2], "rms", m["w_post"], 1.0), 3e-3, "r")
    near(f["z"], ob.front(f["r"], cu, "layer", None, mod[:, 4], mod[:, 3]), 3e-3, "z")
    ref = ob.block_norm_bwd(f["r"], cu, m["dr"], m["dz"], y=f["y"], gate=mod[:, 2], post="rms", w_post=m["w_post"],
                            pre="layer", scale=mod[:, 4], shift=mod[:, 3])
    for name in ("dx", "dy", "dgate", "dscale", "dshift", "dw_post"):
        near(b["join"][name], ref[name], 3e-3, name)
    refs = ob.sparse_attention_bwd(f["q"], f["k"], f["v"], f["o"], f["lse"], b["do"], cu, ri, rc, D ** -0.5)
    for name, r in zip(("dq", "dk", "dv"), refs):
        near(b[name], r, 1e-2, name)
    near(b["dqr"], ob.rope_axes(b["dq"], m["pos"], DIMS, THETA, inverse=True), 3e-3, "dq before the rotation")
    near(b["dkr"], ob.rope_axes(b["dk"], m["pos"], DIMS, THETA, inverse=True), 3e-3, "dk before the rotation")


def test_block_gradient_against_differences(cuda_device):
    """The gradient of the whole chain along random directions of x and of the modulation, against central differences
    of the fp64 chain with the GPU's selection: within 2 % (some ten bf16 roundings stand between them, each 2^-9 of a
    value in the mean and of random sign)."""
    m = _model(2)
    f = _forward(_gpu(m, cuda_device))
    b = _backward(_gpu(m, cuda_device), f)
    idx, cnt, cu = f["idx"].cpu().numpy(), f["cnt"].cpu().numpy(), m["cu"].numpy()
    w = {k: ob.f64(m[k]) for k in ("x", "mod", "w_qkv", "w_o", "w_post", "dr", "dz")}

    def loss(x, mod):
        T = len(x)
        h = ob.front(x, cu, "layer", None, mod[:, 1], mod[:, 0])
        qkv = (h @ w["w_qkv"].T).reshape(T, 3, H, D)
        q, k = (ob.rope_axes(qkv[:, i], m["pos"], DIMS, THETA) for i in range(2))
        o, _ = ob.sparse_attention(q, k, qkv[:, 2], cu, idx, cnt, D ** -0.5)
        y = o.reshape(T, -1) @ w["w_o"].T
        r = ob.join(x, cu, y, mod[:, 2], "rms", w["w_post"], 1.0)
        z = ob.front(r, cu, "layer", None, mod[:, 4], mod[:, 3])
        return (w["dr"] * r).sum() + (w["dz"] * z).sum()

    rng = np.random.default_rng(3)
    zero = np.zeros((len(LENS), C))
    dmod = np.stack([_f(b["front"]["dshift"]), _f(b["front"]["dscale"]), _f(b["join"]["dgate"]),
                     _f(b["join"]["dshift"]), _f(b["join"]["dscale"]), zero], 1)
    dx = _f(b["dx"])
    for _ in range(2):
        u, v = rng.normal(size=w["x"].shape), rng.normal(size=w["mod"].shape)
        v[:, 5] = 0
        e = 1e-4
        want_x = (loss(w["x"] + e * u, w["mod"]) - loss(w["x"] - e * u, w["mod"])) / (2 * e)
        want_m = (loss(w["x"], w["mod"] + e * v) - loss(w["x"], w["mod"] - e * v)) / (2 * e)
        # a random direction's derivative is of the gradient's norm
        assert abs((dx * u).sum() - want_x) <= 0.02 * np.linalg.norm(dx)
        assert abs((dmod * v).sum() - want_m) <= 0.02 * np.linalg.norm(dmod)


def test_block_captured_and_on_two_streams(cuda_device):
    """The chain captured into a graph, replayed with new inputs, and two chains at once on streams of their own."""
    m1, m2 = _gpu(_model(4), cuda_device), _gpu(_model(5), cuda_device)
    want = [_forward(m) for m in (m1, m2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [_forward(m, s) for m, s in zip((m1, m2), streams)]
    assert all(pa.pa_get_error(s) == pa.PA_OK for s in streams)
    for a, w in zip(got, want):
        assert all(torch.equal(a[k], w[k]) for k in w)
    static = {k: v.clone() for k, v in m1.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _forward(static)
    for m, w in ((m2, want[1]), (m1, want[0])):
        for k in static:
            static[k].copy_(m[k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], w[k]) for k in w)
