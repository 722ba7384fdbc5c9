"""Infinities and NaN in the block operators: they reach what the formulas say they reach, and nothing else.

The oracle says where an output is NaN; no tolerance enters.  Everything a NaN does not reach is compared bit by bit
with the same call on finite inputs.
"""
import numpy as np
import pytest
import torch

import dit_resolution_packed_b200 as pa
import workloads
from oracle import block as ob

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
SUMS = ("dgate", "dscale", "dshift", "dw_post", "dw_pre")


def _inputs(lens, C, f32, seed):
    g = torch.Generator().manual_seed(seed)
    wide = torch.float32 if f32 else torch.bfloat16
    T, B = sum(lens), len(lens)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32), x=rn(T, C).to(wide),
             y=rn(T, C).to(torch.bfloat16), dr=rn(T, C).to(wide), dz=rn(T, C).to(torch.bfloat16))
    m = (0.3 * rn(3, B, C)).to(wide)
    t["gate"], t["scale"], t["shift"] = m[0].clone(), m[1].clone(), m[2].clone()
    t["w_post"], t["w_pre"] = ((1 + 0.2 * rn(C)).to(wide) for _ in range(2))
    return t


def _run(dev, t, post, pre):
    """(r, z, gradients) on the GPU, with the oracle's of the stored r."""
    d = {k: v.to(dev) for k, v in t.items()}
    how = dict(y=d["y"], gate=d["gate"], post=post, w_post=d["w_post"], pre=pre, w_pre=d["w_pre"], scale=d["scale"],
               shift=d["shift"])
    r, z = pa.block_norm_fwd(d["x"], d["cu"], **how)
    out = pa.block_norm_bwd(r, d["cu"], d["dr"], d["dz"], **how)
    assert pa.pa_get_error() == pa.PA_OK
    cu = t["cu"].numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        ref = ob.block_norm_bwd(r, cu, t["dr"], t["dz"], y=t["y"], gate=t["gate"], post=post, w_post=t["w_post"],
                                pre=pre, w_pre=t["w_pre"], scale=t["scale"], shift=t["shift"])
        ref["r"] = ob.join(t["x"], cu, t["y"], t["gate"], post, t["w_post"], 1.0)
        ref["z"] = ob.front(r, cu, pre, t["w_pre"], t["scale"], t["shift"])
    return dict(out, r=r, z=z), ref


def _same_nans(got, ref, names, what):
    for name in names:
        assert np.array_equal(torch.isnan(got[name].float()).cpu().numpy(), np.isnan(ref[name])), f"{what}: {name}"


# one, two and four warps a row forward; one team of each width backward
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("C", [72, 512, 2560, 4096])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("rms", "layer"), ("layer", "rms"), ("layer", "layer")])
@pytest.mark.parametrize("where", ["x", "y", "dr", "dz"])
def test_a_nan_reaches_its_row(cuda_device, where, post, pre, C, f32):
    t = _inputs([40, 30], C, f32, 1)
    clean, _ = _run(cuda_device, t, post, pre)
    row, channel = 57, C - 3
    t[where][row, channel] = NAN
    got, ref = _run(cuda_device, t, post, pre)
    _same_nans(got, ref, ("r", "z", "dx", "dy") + SUMS, f"NaN in {where}")
    keep = torch.arange(70, device=cuda_device) != row
    for name in ("r", "z", "dx", "dy"):
        assert torch.equal(got[name][keep], clean[name][keep]), name
    for name in ("dgate", "dscale", "dshift"):
        assert torch.equal(got[name][0], clean[name][0]), name


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("C", [72, 512, 2560, 4096])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("channel", [0, -1])  # inside and behind the channels that a row's pivot is taken from
def test_an_infinity_reaches_its_row(cuda_device, channel, kind, C, f32):
    """Forward: a layer norm's whole row is NaN; an rms norm's is 0, and NaN where the infinity stands."""
    t = _inputs([40, 30], C, f32, 2)
    for where in ("x", "y"):
        s = dict(t, **{where: t[where].clone()})
        s[where][7, channel] = -INF
        got, ref = _run(cuda_device, s, kind, kind)
        _same_nans(got, ref, ("r", "z"), f"infinity in {where}")
        name = "z" if where == "x" else "r"
        nan = np.isnan(ref[name][7])
        assert nan.all() if kind == "layer" else nan.sum() == 1


def _bits(x):
    return x.cpu().view(torch.int16)


def _odd_values(x, channels):
    """Infinities, NaN and a negative zero in some of the given channels of every third token."""
    x = x.clone()
    for i, v in enumerate((INF, NAN, -INF, -0.0)):
        x[i::3, :, channels[i % len(channels)]] = v
    return x


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,dims", [(64, [8, 16]), (64, [62]), (128, [6, 50]), (128, [32]), (128, [2, 2, 2])])
def test_channels_behind_the_axes_are_copied_whatever_they_hold(cuda_device, d, dims, inter):
    g = torch.Generator().manual_seed(3)
    T, H, n = 50, 3, sum(dims) // 2
    rest = list(range(2 * n, d)) if inter else list(range(n, d // 2)) + list(range(d // 2 + n, d))
    turned = [c for c in range(d) if c not in rest]
    pos = torch.floor(torch.rand(T, len(dims), generator=g) * 40).to(cuda_device)
    clean = [torch.randn(T, H, d, generator=g).to(torch.bfloat16) for _ in range(2)]
    odd = [_odd_values(x, rest[1::2] or rest) for x in clean]
    for fn in (pa.rope_axes_fwd, pa.rope_axes_bwd):
        want = fn(*(x.to(cuda_device) for x in clean), pos, dims, 100.0, inter)
        got = fn(*(x.to(cuda_device) for x in odd), pos, dims, 100.0, inter)
        for a, b, x in zip(got, want, odd):
            assert torch.equal(_bits(a)[..., rest], x.view(torch.int16)[..., rest])
            assert torch.equal(a[..., turned], b[..., turned])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,dims", [(64, [8, 16]), (64, [62]), (128, [6, 50]), (128, [32])])
def test_the_projection_leaves_channels_behind_the_axes(cuda_device, d, dims, inter):
    """They are what the linear layer gives, also beside an infinity."""
    g = torch.Generator().manual_seed(4)
    T, C, H, n = 150, 72, 3, sum(dims) // 2
    rest = list(range(2 * n, d)) if inter else list(range(n, d // 2)) + list(range(d // 2 + n, d))
    x = torch.randn(T, C, generator=g).to(torch.bfloat16).to(cuda_device)
    w = (torch.randn(3, H, d, C, generator=g) * C ** -0.5).to(torch.bfloat16)
    w[:, 1, rest[-1], 5] = INF
    w = w.view(3 * H * d, C).to(cuda_device)
    pos = torch.floor(torch.rand(T, len(dims), generator=g) * 40).to(cuda_device)
    q, k, v = pa.qkv_rope_axes_fwd(x, w, pos, H, d, dims, 100.0, inter)
    y = pa.linear_fwd(x, w).view(T, 3, H, d)
    assert torch.equal(_bits(v.contiguous()), _bits(y[:, 2].contiguous()))
    for i, got in enumerate((q, k)):
        assert torch.equal(_bits(got)[..., rest], _bits(y[:, i].contiguous())[..., rest])


@pytest.mark.parametrize("lens", [[0, 40, 0, 30, 0], [1] * 50 + [0] * 20])  # both ways of adding an image's sums
def test_factors_of_images_without_tokens_have_no_effect(cuda_device, lens):
    """Rows of the modulation behind the last image of a padded batch may hold anything."""
    t = _inputs(lens, 264, False, 5)
    t["w_pre"][3] = INF
    t["w_post"][5] = -INF
    clean, _ = _run(cuda_device, t, "rms", "layer")
    empty = [s for s, n in enumerate(lens) if n == 0]
    for name, v in (("gate", NAN), ("scale", INF), ("shift", NAN)):
        t[name][empty] = v
    got, _ = _run(cuda_device, t, "rms", "layer")
    for name in clean:
        assert np.array_equal(*(x[name].float().cpu().numpy() for x in (got, clean)), equal_nan=True), name
    for name in ("dgate", "dscale", "dshift"):
        assert not got[name][empty].any(), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["q", "k", "v", "dout"])
def test_attention_over_a_listed_key_that_is_not_finite(cuda_device, where, value, d):
    """NaN where the formulas give it, whichever key of a tile it is (some exponentials are polynomials), in the first tile
    of a row and in later ones; the dense calls too."""
    lens, H, row_blocks = [300, 40], 2, 3
    p = workloads.random_pack(lens, H, d, 41)
    clean = {n: p[n] for n in ("q", "k", "v")}
    clean["dout"] = workloads.random_dout(p["q"].shape, 42)
    cu, rows = p["cu_seqlens"], ob.table_rows(2, 340)
    cnt = torch.zeros(H, rows, dtype=torch.int32)
    idx = torch.arange(row_blocks, dtype=torch.int32).repeat(H, rows, 1)
    for s, n in enumerate(lens):
        first = ob.first_row(cu.numpy(), s)
        cnt[:, first:first + ob.n_blocks(n)] = ob.n_blocks(n)
    gc, gi, gn = cu.to(cuda_device), idx.to(cuda_device), cnt.to(cuda_device)
    scale = d ** -0.5
    g = {n: x.to(cuda_device) for n, x in clean.items()}
    out, lse = pa.block_sparse_attn_fwd(g["q"], g["k"], g["v"], gc, 300, gi, gn)
    for at in list(range(8)) + [133, 262]:
        t = dict(clean, **{where: clean[where].clone()})
        t[where][at, 0, 5] = value
        g = {n: x.to(cuda_device) for n, x in t.items()}
        runs = [(pa.block_sparse_attn_fwd(g["q"], g["k"], g["v"], gc, 300, gi, gn),
                 pa.block_sparse_attn_bwd(g["q"], g["k"], g["v"], out, lse, g["dout"], gc, 300, gi, gn)),
                (pa.varlen_attn_fwd(g["q"], g["k"], g["v"], gc, 300),
                 pa.varlen_attn_bwd(g["q"], g["k"], g["v"], out, lse, g["dout"], gc, 300))]
        assert pa.pa_get_error() == pa.PA_OK
        # the oracle of the first image alone, whose every pair is visible: over the whole pack its matrix products would
        # take 0 times NaN for the pairs of different images
        one = [t[n][:300] for n in ("q", "k", "v")]
        lists = np.array([0, 300]), idx[:, :3].numpy(), cnt[:, :3].numpy(), scale
        with np.errstate(all="ignore"):
            want = ob.sparse_attention(*one, *lists)
            want += ob.sparse_attention_bwd(*one, out[:300], lse[:300], t["dout"][:300], *lists)
        for form, got in zip(("sparse", "dense"), runs):
            for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got[0] + got[1], want):
                nan = torch.isnan(a.float()).cpu().numpy()
                assert np.array_equal(nan[:300], np.isnan(b)) and not nan[300:].any(), f"{form} {name}, token {at}"
