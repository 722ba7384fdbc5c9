"""Gated residual join with its norms (pa_block_norm_fwd, pa_block_norm_bwd) on the GPU vs the fp64 oracle.

Tolerances, from the arithmetic: an output rounded to bf16 is off by half a step (2^-8 of its value).  The fp32
part before it: every sum over a row of C channels runs through chains of at most 8 + 5 + 32 additions, and a few
more operations follow, so each term of a formula is off by at most 64 x 2^-24 of the magnitudes that enter it
(hat: of |v| and mean |v|, over the deviation).  Column sums over n tokens go through chains of at most
64 + n / 512 + 8 additions.  `unit` below is that count with a factor 4 for the operations per term.
"""
import numpy as np
import pytest
import torch

import dit_resolution_packed_b200 as pa
from oracle import block as ob

pytestmark = pytest.mark.gpu
EPS32 = 2.0 ** -24
UNIT = 256 * EPS32
HALF = 2.0 ** -8


def _case(lens, C, f32, seed, join=True, mod=True, weights=True, offset=0.0, pf32=None):
    g = torch.Generator().manual_seed(seed)
    wide = torch.float32 if f32 else torch.bfloat16
    param = wide if pf32 is None else (torch.float32 if pf32 else torch.bfloat16)
    T, B = sum(lens), len(lens)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    chan = torch.exp(0.5 * rn(C))
    t = dict(cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32),
             x=(rn(T, C) * chan + offset).to(wide), y=(rn(T, C) + offset).to(torch.bfloat16) if join else None,
             dr=rn(T, C).to(wide), dz=rn(T, C).to(torch.bfloat16))
    m = (0.3 * rn(B, 3, C)).to(param)
    t["gate"], t["scale"], t["shift"] = (m[:, 0] if join else None, m[:, 1], m[:, 2]) if mod else (None,) * 3
    w = [(1 + 0.2 * rn(C)).to(param) for _ in range(2)]
    t["w_post"], t["w_pre"] = (w[0] if join else None, w[1]) if weights else (None, None)
    return t


def _on(t, dev):
    names = [n for n in ("gate", "scale", "shift") if t[n] is not None]
    if names:  # keep the slices of one projection strided
        m = torch.stack([t[n] for n in names], 1).to(dev)
        t = dict(t, **{n: m[:, i] for i, n in enumerate(names)})
    return {k: v.to(dev) if torch.is_tensor(v) and v.device.type == "cpu" else v for k, v in t.items()}


def _within(got, ref, bound, what):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    worst = float(np.max(np.abs(got - ref) / bound)) if ref.size else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} past the bound, worst {worst:.2f}"


def _out_err(ref, wide):
    return np.abs(ref) * (HALF if wide == torch.bfloat16 else EPS32) * (1 + HALF) + 1e-30


def _hat_size(v, kind):
    """|v| and mean |v| over the deviation: what the error of a normed value scales with."""
    if kind == "none":
        return np.abs(v)
    hat, rstd = ob.normed(v, kind, 1e-6)
    return rstd * (np.abs(v) + np.abs(v).mean(-1, keepdims=True)) + np.abs(hat)


def _check_fwd(t, r, z, post, pre, res):
    cu, (T, C) = t["cu"].cpu().numpy(), t["x"].shape
    seg = ob.segment_ids(cu, T)
    if t["y"] is not None:
        ref = ob.join(t["x"], cu, t["y"], t["gate"], post, t["w_post"], res)
        g = np.abs(ob._rows(t["gate"], seg, 1.0, (T, C)) * ob._vec(t["w_post"], C))
        _within(r, ref, _out_err(ref, t["x"].dtype) + UNIT * (np.abs(res * ob.f64(t["x"]))
                                                              + g * _hat_size(ob.f64(t["y"]), post)), "r")
    if pre != "none":
        ref = ob.front(r, cu, pre, t["w_pre"], t["scale"], t["shift"])
        a = np.abs(ob._vec(t["w_pre"], C) * (1 + ob._rows(t["scale"], seg, 0.0, (T, C))))
        _within(z, ref, _out_err(ref, torch.bfloat16) + UNIT * (
            a * _hat_size(ob.f64(r), pre) + np.abs(ob._rows(t["shift"], seg, 0.0, (T, C)))), "z")


def _check_bwd(t, r, out, post, pre, res, dr=True):
    cu, (T, C) = t["cu"].cpu().numpy(), t["x"].shape
    seg = ob.segment_ids(cu, T)
    how = dict(y=t["y"], gate=t["gate"], post=post, w_post=t["w_post"], res=res, pre=pre, w_pre=t["w_pre"],
               scale=t["scale"], shift=t["shift"])
    ref = ob.block_norm_bwd(r, cu, t["dr"] if dr else None, t["dz"] if pre != "none" else None, **how)
    mag = np.abs(ob.f64(t["dr"])) if dr else np.zeros((T, C))
    if pre != "none":
        dz, rr = np.abs(ob.f64(t["dz"])), ob.f64(r)
        hat, rstd = ob.normed(rr, pre, 1e-6)
        size = _hat_size(rr, pre)
        a = np.abs(ob._vec(t["w_pre"], C) * (1 + ob._rows(t["scale"], seg, 0.0, (T, C))))
        gm = dz * a
        mag = mag + rstd * (gm + gm.mean(1, keepdims=True) + size * (gm * size).mean(1, keepdims=True))
    _within(out["dx"], ref["dx"], _out_err(ref["dx"], t["x"].dtype) + UNIT * res * mag, "dx")

    def by_seg(v):
        s = np.zeros((len(cu) - 1, C))
        np.add.at(s, seg, v)
        return s

    longest = UNIT * (1 + T / 4096.0)
    if pre != "none":
        w = np.abs(ob._vec(t["w_pre"], C))
        if t["scale"] is not None:
            _within(out["dscale"], ref["dscale"], longest * by_seg(dz * size * w) + 1e-30, "dscale")
            _within(out["dshift"], ref["dshift"], longest * by_seg(dz) + 1e-30, "dshift")
        if t["w_pre"] is not None:
            up = np.abs(1 + ob._rows(t["scale"], seg, 0.0, (T, C)))
            _within(out["dw_pre"], ref["dw_pre"], longest * (dz * up * size).sum(0) + 1e-30, "dw_pre")
    if t["y"] is not None:
        y = ob.f64(t["y"])
        size = _hat_size(y, post)
        _, rstd = ob.normed(y, post, 1e-6)
        g = np.abs(ob._rows(t["gate"], seg, 1.0, (T, C)) * ob._vec(t["w_post"], C))
        gm = mag * g
        dym = gm if post == "none" else rstd * (gm + gm.mean(1, keepdims=True) + size * (gm * size).mean(1, keepdims=True))
        _within(out["dy"], ref["dy"], _out_err(ref["dy"], torch.bfloat16) + UNIT * dym, "dy")
        if t["gate"] is not None:
            _within(out["dgate"], ref["dgate"], longest * by_seg(mag * size * np.abs(ob._vec(t["w_post"], C))) + 1e-30,
                    "dgate")
        if t["w_post"] is not None:
            gate = np.abs(ob._rows(t["gate"], seg, 1.0, (T, C)))
            _within(out["dw_post"], ref["dw_post"], longest * (mag * gate * size).sum(0) + 1e-30, "dw_post")


def _run(dev, t, post, pre, res=1.0, dr=True):
    d = _on(t, dev)
    how = dict(y=d["y"], gate=d["gate"], post=post, w_post=d["w_post"], residual_scale=res, pre=pre, w_pre=d["w_pre"],
               scale=d["scale"], shift=d["shift"])
    r, z = pa.block_norm_fwd(d["x"], d["cu"], **how)
    out = pa.block_norm_bwd(r, d["cu"], d["dr"] if dr else None, d["dz"] if pre != "none" else None, **how)
    assert pa.pa_get_error() == pa.PA_OK
    _check_fwd(t, r, z, post, pre, res)
    _check_bwd(t, r, out, post, pre, res, dr)
    return r, z, out


LENS = [3, 0, 130, 1, 64, 0]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("C", [520, 1152, 1536, 1800, 2304, 2312, 2560, 3080, 3584, 4088, 4096, 5120, 5128, 6144, 6152, 7168, 7176])
def test_channels_of_every_split(cuda_device, C, f32):
    """Every number of warps that a row, a team and a block can have, with all four tensors in the rows."""
    _run(cuda_device, _case([70, 9], C, f32, 14), "layer", "layer")
    _run(cuda_device, _case([33], C, f32, 15, join=False), "none", "rms", dr=False)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("C", [8, 72, 256, 264, 1032, 2048, 2056, 4104, 8192])
def test_channels(cuda_device, C, f32):
    _run(cuda_device, _case(LENS, C, f32, 1), "rms", "layer")


@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("pre", ["none", "layer", "rms"])
@pytest.mark.parametrize("mod,weights", [(True, True), (True, False), (False, True), (False, False)])
def test_kinds(cuda_device, post, pre, mod, weights):
    t = _case(LENS, 320, False, 2, mod=mod, weights=weights)
    if pre == "none":
        t.update(scale=None, shift=None, w_pre=None)
    _run(cuda_device, t, post, pre, res=0.5)


@pytest.mark.parametrize("f32", [False, True])
def test_norm_alone(cuda_device, f32):
    t = _case(LENS, 520, f32, 3, join=False)
    r, _, _ = _run(cuda_device, t, "none", "layer", dr=False)
    assert torch.equal(r.cpu(), t["x"])


def test_parameters_of_the_other_type(cuda_device):
    _run(cuda_device, _case(LENS, 136, True, 4, pf32=False), "rms", "layer")
    _run(cuda_device, _case(LENS, 136, False, 5, pf32=True), "rms", "layer")


@pytest.mark.parametrize("lens", [[1], [0, 0, 5], [1] * 700, [4500, 3, 700]])
def test_packs(cuda_device, lens):
    _run(cuda_device, _case(lens, 264, False, 6), "layer", "rms")


def test_mean_far_above_the_deviation(cuda_device):
    """The statistics do not cancel: rows whose mean is 2000 times their deviation."""
    t = _case([70], 2048, True, 7, offset=0.0, mod=False, weights=False)
    t["x"] = t["x"] * 0.5 + 1000.0
    t["y"] = torch.zeros_like(t["y"])
    _run(cuda_device, t, "none", "layer")


def test_constant_and_nan_rows_stay_apart(cuda_device):
    """A row of zeros has deviation sqrt(eps); a NaN row leaves every other row alone."""
    t = _case([40, 40], 512, False, 8)
    t["x"][5] = 0
    t["y"][5] = 0
    clean = _run(cuda_device, t, "rms", "layer")
    t["x"][60, 3] = float("nan")
    d = _on(t, cuda_device)
    r, z = pa.block_norm_fwd(d["x"], d["cu"], y=d["y"], gate=d["gate"], post="rms", w_post=d["w_post"], pre="layer",
                             w_pre=d["w_pre"], scale=d["scale"], shift=d["shift"])
    keep = torch.arange(80) != 60
    assert torch.isnan(z[60].float()).all()
    assert torch.equal(r.cpu()[keep], clean[0].cpu()[keep]) and torch.equal(z.cpu()[keep], clean[1].cpu()[keep])


def test_no_tokens_gives_zero_sums(cuda_device):
    t = _case([0, 0], 64, False, 9)
    d = _on(t, cuda_device)
    out = pa.block_norm_bwd(d["x"], d["cu"], d["dr"], d["dz"], y=d["y"], gate=d["gate"], post="rms",
                            w_post=d["w_post"], pre="layer", w_pre=d["w_pre"], scale=d["scale"], shift=d["shift"])
    for name in ("dgate", "dscale", "dshift", "dw_post", "dw_pre"):
        assert not out[name].any(), name


def test_one_row_of_factors_for_all_images(cuda_device):
    """A broadcast gate (row stride 0): its gradient comes per image, to be summed by the caller."""
    t = _case([30, 50], 128, False, 10)
    row = t["gate"][:1].clone()
    t["gate"] = row.expand(2, 128)
    d = {k: v.to(cuda_device) if torch.is_tensor(v) else v for k, v in t.items()}
    d["gate"] = row.to(cuda_device).expand(2, 128)
    for name in ("scale", "shift"):
        d[name] = d[name].contiguous()
    how = dict(y=d["y"], gate=d["gate"], post="rms", w_post=d["w_post"], pre="layer", w_pre=d["w_pre"],
               scale=d["scale"], shift=d["shift"])
    assert d["gate"].stride(0) == 0
    r, z = pa.block_norm_fwd(d["x"], d["cu"], **how)
    out = pa.block_norm_bwd(r, d["cu"], d["dr"], d["dz"], **how)
    _check_fwd(t, r, z, "rms", "layer", 1.0)
    _check_bwd(t, r, out, "rms", "layer", 1.0)


def test_in_place_and_repeatable(cuda_device):
    t = _case([100, 300], 1152, True, 11)
    d = _on(t, cuda_device)
    how = dict(gate=d["gate"], post="rms", w_post=d["w_post"], pre="layer", w_pre=d["w_pre"], scale=d["scale"],
               shift=d["shift"])
    r, z = pa.block_norm_fwd(d["x"], d["cu"], y=d["y"], **how)
    a = pa.block_norm_bwd(r, d["cu"], d["dr"], d["dz"], y=d["y"], **how)
    b = pa.block_norm_bwd(r, d["cu"], d["dr"], d["dz"], y=d["y"], **how)
    assert all(torch.equal(a[k], b[k]) for k in a)
    x2, z2 = d["x"].clone(), torch.empty_like(z)
    assert pa.pa_block_norm_fwd(x2, d["cu"], d["y"], x2, z2, **how) == pa.PA_OK
    assert torch.equal(x2, r) and torch.equal(z2, z)
    g = d["dr"].clone()
    ws = torch.empty(pa.pa_block_norm_workspace_bytes(2, 400, 1152), dtype=torch.uint8, device=cuda_device)
    dy = torch.empty_like(d["y"])
    assert pa.pa_block_norm_bwd(r, d["cu"], d["y"], g, d["dz"], g, dy, a["dgate"], None, None, None, None, ws,
                                **how) == pa.PA_OK
    assert torch.equal(g, b["dx"]) and torch.equal(dy, b["dy"]) and torch.equal(a["dgate"], b["dgate"])


def test_streams_and_graphs(cuda_device):
    """Another stream, and two captured graphs with scratch of their own replayed at once."""
    t = _case([257, 300], 520, False, 12)
    d = _on(t, cuda_device)
    how = dict(y=d["y"], gate=d["gate"], post="rms", w_post=d["w_post"], pre="layer", w_pre=d["w_pre"],
               scale=d["scale"], shift=d["shift"])
    r, z = pa.block_norm_fwd(d["x"], d["cu"], **how)
    want = pa.block_norm_bwd(r, d["cu"], d["dr"], d["dz"], **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2, z2 = pa.block_norm_fwd(d["x"], d["cu"], stream=side, **how)
    got = pa.block_norm_bwd(r2, d["cu"], d["dr"], d["dz"], stream=side, **how)
    assert pa.pa_get_error(side) == pa.PA_OK
    assert torch.equal(z2, z) and all(torch.equal(got[k], want[k]) for k in want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rg, zg = pa.block_norm_fwd(d["x"], d["cu"], **how)
            og = pa.block_norm_bwd(rg, d["cu"], d["dr"], d["dz"], **how)
        graphs.append((g, zg, og))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, zg, og), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                zg.zero_()
                g.replay()
    torch.cuda.synchronize()
    for _, zg, og in graphs:
        assert torch.equal(zg, z) and all(torch.equal(og[k], want[k]) for k in want)


def test_bad_cu_seqlens_is_recorded(cuda_device):
    t = _case([10, 20], 64, False, 13)
    d = _on(t, cuda_device)
    for bad in ([0, 25, 20], [0, 10, 29], [1, 10, 30], [0, -7, 30]):
        cu = torch.tensor(bad, dtype=torch.int32, device=cuda_device)
        pa.block_norm_fwd(d["x"], cu, y=d["y"], gate=d["gate"], pre="layer")
        assert pa.pa_get_error() == pa.PA_ERR_CU_SEQLENS
        pa.block_norm_bwd(d["x"], cu, d["dr"], d["dz"], y=d["y"], gate=d["gate"], pre="layer")
        assert pa.pa_get_error() == pa.PA_ERR_CU_SEQLENS


@pytest.mark.parametrize("C", [72, 264, 520, 1152, 2056])
@pytest.mark.parametrize("lens", [[2500] + [3] * 45, [3] * 30 + [0, 1500] + [1] * 12 + [0, 1200, 0],
                                  [10, 75] * 30, [180] * 41])
def test_long_images_among_many(cuda_device, lens, C):
    """More images than the sums take one by one, some of them over many runs of rows."""
    _run(cuda_device, _case(lens, C, False, 16), "rms", "layer")
