"""Pins of the oracle of the block around the attention (``oracle/block.py``): closed forms, the dense oracle, torch's
own norms, and every gradient against central differences."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import block as ob

RNG = np.random.default_rng(5)


def _difference(f, x, at, h=1e-5):
    x1, x2 = x.copy(), x.copy()
    x1[at] += h
    x2[at] -= h
    return (f(x1) - f(x2)) / (2 * h)


def _entries(shape, n=6):
    return [tuple(int(RNG.integers(0, s)) for s in shape) for _ in range(n)]


def test_norms_match_torch():
    v = torch.from_numpy(RNG.normal(2.0, 3.0, (5, 24)))
    assert np.allclose(ob.normed(v.numpy(), "layer", 1e-6)[0], torch.nn.functional.layer_norm(v, (24,), eps=1e-6),
                       atol=1e-13)
    assert np.allclose(ob.normed(v.numpy(), "rms", 1e-6)[0], torch.nn.functional.rms_norm(v, (24,), eps=1e-6),
                       atol=1e-13)
    assert ob.normed(v.numpy(), "none", 1e-6)[0] is not None


@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "rms"), ("layer", "layer"), ("layer", "none")])
def test_norm_gradients_match_differences(post, pre):
    cu, C = [0, 3, 3, 7], 16
    T, B = 7, 3
    a = dict(x=RNG.normal(size=(T, C)), y=RNG.normal(size=(T, C)), gate=RNG.normal(size=(B, C)),
             scale=RNG.normal(size=(B, C)), shift=RNG.normal(size=(B, C)), w_post=RNG.normal(size=C),
             w_pre=RNG.normal(size=C))
    dr, dz, res = RNG.normal(size=(T, C)), RNG.normal(size=(T, C)), 0.7

    def loss(**kw):
        b = dict(a, **kw)
        r = ob.join(b["x"], cu, b["y"], b["gate"], post, b["w_post"], res)
        total = (dr * r).sum()
        if pre != "none":
            total += (dz * ob.front(r, cu, pre, b["w_pre"], b["scale"], b["shift"])).sum()
        return total

    r = ob.join(a["x"], cu, a["y"], a["gate"], post, a["w_post"], res)
    grads = ob.block_norm_bwd(r, cu, dr, dz if pre != "none" else None, y=a["y"], gate=a["gate"], post=post,
                              w_post=a["w_post"], res=res, pre=pre, w_pre=a["w_pre"], scale=a["scale"],
                              shift=a["shift"])
    names = ["x", "y", "gate", "w_post"] + (["scale", "shift", "w_pre"] if pre != "none" else [])
    for name in names:
        got = grads["d" + name]
        for at in _entries(got.shape):
            want = _difference(lambda v: loss(**{name: v}), a[name], at)
            assert abs(got[at] - want) <= 1e-6 * (1 + abs(want)), (name, at)
    assert not grads["dgate"][1].any()  # the empty image


def test_rope_properties():
    T, H, d, dims = 9, 2, 64, [16, 24, 24]
    x, pos = RNG.normal(size=(T, H, d)), RNG.normal(size=(T, 3)) * 50
    for inter in (False, True):
        y = ob.rope_axes(x, pos, dims, 100.0, inter)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.allclose(ob.rope_axes(y, pos, dims, 100.0, inter, inverse=True), x)
        assert np.allclose(ob.rope_axes(x, pos * 0, dims, 100.0, inter), x)
        # products depend on the difference of the positions alone
        q, k = x[:1], x[1:2]
        shift = np.array([[3.0, -2.0, 5.5]])
        dot = lambda p1, p2: (ob.rope_axes(q, p1, dims, 100.0, inter) * ob.rope_axes(k, p2, dims, 100.0, inter)).sum()  # noqa: E731,B023
        assert abs(dot(pos[:1], pos[1:2]) - dot(pos[:1] + shift, pos[1:2] + shift)) < 1e-9
        # the inverse is the gradient: <dy, R x> = <R' dy, x>
        dy = RNG.normal(size=x.shape)
        assert abs((dy * y).sum() - (ob.rope_axes(dy, pos, dims, 100.0, inter, inverse=True) * x).sum()) < 1e-9
    # channels behind the axes stay
    y = ob.rope_axes(x, pos[:, :1], [16], 100.0, False)
    assert np.array_equal(y[..., 8:32], x[..., 8:32]) and np.array_equal(y[..., 40:], x[..., 40:])
    # one axis over all channels is the projection's rotation
    from oracle import proj
    one = ob.rope_axes(x, np.arange(T)[:, None], [64], 10000.0, False)
    assert np.allclose(one, proj.rope(x, np.arange(T), 10000.0), atol=1e-12)


def test_select_counts_order_and_ties():
    cu = [0, 300, 300, 940]
    q, k = RNG.normal(size=(940, 2, 64)), RNG.normal(size=(940, 2, 64))
    idx, cnt = ob.block_select(q, k, cu, 0.5, 2, 3)
    assert idx.shape == (2, 940 // 128 + 3, 3)
    rows = {0: (0, 3), 2: (300 // 128 + 2, 5)}
    used = np.zeros(idx.shape[1], dtype=bool)
    for s, (row, nb) in rows.items():
        keep = ob.keep_count(cu[s + 1] - cu[s], 0.5, 2)
        assert keep == {0: 2, 2: 3}[s]
        assert (cnt[:, row:row + nb] == keep).all()
        assert (np.diff(idx[:, row:row + nb, :keep], axis=-1) > 0).all()
        assert (idx[:, row:row + nb, keep:] == -1).all()
        used[row:row + nb] = True
    assert (cnt[:, ~used] == 0).all() and (idx[:, ~used] == -1).all()
    # equal scores: the lower block
    idx, _ = ob.block_select(np.zeros((640, 1, 64)), k[:640, :1], [0, 640], 0.4, 1, 2)
    assert (idx[0, :5] == [0, 1]).all()
    # a block whose mean is a NaN ranks last, as -infinity
    bad = k[:640, :1].copy()
    bad[0] = np.nan
    idx, _ = ob.block_select(q[:640, :1], bad, [0, 640], 0.8, 1, 4)
    assert (idx[0, :5] == [1, 2, 3, 4]).all()


def test_all_blocks_is_the_dense_attention():
    cu = [0, 200, 200, 470]
    q, k, v, do = (RNG.normal(size=(470, 2, 64)).astype(np.float32) for _ in range(4))
    idx, cnt = ob.block_select(q, k, cu, 1.0, 1, 3)
    out, lse = ob.sparse_attention(q, k, v, cu, idx, cnt, 0.125)
    to = [torch.from_numpy(x).to(torch.bfloat16) for x in (q, k, v, do)]
    ref_o, ref_l = oracle.varlen_attention(*to[:3], torch.tensor(cu, dtype=torch.int32), 0.125)
    out, lse = ob.sparse_attention(*to[:3], cu, idx, cnt, 0.125)
    assert np.allclose(out, ref_o, atol=1e-12) and np.allclose(lse, ref_l, atol=1e-12)
    refs = oracle.varlen_attention_bwd(*to, torch.tensor(cu, dtype=torch.int32), 0.125)
    got = ob.sparse_attention_bwd(*to[:3], out, lse, to[3], cu, idx, cnt, 0.125)
    for a, b in zip(got, refs):
        assert np.allclose(a, b, atol=1e-10)


def test_sparse_gradients_match_differences_and_empty_rows():
    cu, T = [0, 150, 420], 420
    arr = dict(zip("qkv", (RNG.normal(size=(T, 1, 8)) for _ in range(3))))
    do = RNG.normal(size=(T, 1, 8))
    idx, cnt = ob.block_select(arr["q"], arr["k"], cu, 0.5, 1, 2)
    cnt = cnt.copy()
    cnt[0, 0] = 0  # the first block of queries sees nothing
    idx[0, ob.first_row(cu, 1):ob.first_row(cu, 1) + 3, :2] = [0, 2]  # nobody sees block 1 of the second image

    def loss(**kw):
        b = dict(arr, **kw)
        return (do * ob.sparse_attention(b["q"], b["k"], b["v"], cu, idx, cnt, 0.3)[0]).sum()

    out, lse = ob.sparse_attention(arr["q"], arr["k"], arr["v"], cu, idx, cnt, 0.3)
    assert not out[:128].any() and np.isneginf(lse[:128]).all() and np.isfinite(lse[128:]).all()
    grads = ob.sparse_attention_bwd(arr["q"], arr["k"], arr["v"], out, lse, do, cu, idx, cnt, 0.3)
    assert not grads[0][:128].any() and not grads[1][278:406].any() and not grads[2][278:406].any()
    for name, got in zip("qkv", grads):
        for at in _entries(got.shape, 8):
            want = _difference(lambda x: loss(**{name: x}), arr[name], at)
            assert abs(got[at] - want) <= 1e-6 * (1 + abs(want)), (name, at)


def test_keep_count():
    assert ob.keep_count(1280, 0.1, 1) == 1 and ob.keep_count(1281, 0.1, 1) == 2
    assert ob.keep_count(100, 0.0, 5) == 1 and ob.keep_count(0, 1.0, 1) == 0
    assert ob.keep_count(128 * 7, 0.0, 3) == 3 and math.ceil(0.5 * 7) == ob.keep_count(128 * 7, 0.5, 3)
