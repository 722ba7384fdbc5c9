"""Selection of key blocks and the attention over them (pa_block_select, pa_block_sparse_attn_fwd / _bwd) on the GPU vs
the fp64 oracle.

Tolerances, from the arithmetic (p the exact weights of a row, A B the products of the magnitudes):
  selection   equal: the kernel and the oracle both order fp64 scores;
  out         the softmax weights are rounded to bf16 (half a step, 2^-8 of each) and normalised by their own sum, so
              the value is off by at most 2^-8 sum p |v - out| <= 2^-8 (p |v| + |out|), and out is rounded once more
              (2^-8 |out|); exponentials by polynomial are within 1e-4;
  lse         1e-4 of the exponentials, fp32 scores and sums: 2e-4;
  dv          P rounded to bf16: 2^-8 P'|dout|, dv rounded: 2^-8 |dv|, P itself within 1e-4;
  dq, dk      dS rounded to bf16: 2^-8 |dS| |k| (|q|), the result 2^-8 of itself; dS = scale P (dout v - D) is a
              difference of fp32 sums, within 1e-4 of scale P (|dout||v| + |dout||out|).
"""
import numpy as np
import pytest
import torch

import dit_resolution_packed_b200 as pa
import workloads
from oracle import block as ob

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
EXP = 1e-4


def _inputs(lens, H, d, seed):
    p = workloads.random_pack(lens, H, d, seed)
    dout = workloads.random_dout(p["q"].shape, seed + 1)
    return p["q"], p["k"], p["v"], dout, p["cu_seqlens"], max(lens)


def _bounds(q, k, v, out, lse, dout, cu, idx, cnt, scale):
    """Per head: (out, dq, dk, dv) bounds, from the oracle's own weights."""
    q, k, v, out, lse, dout = (ob.f64(t) for t in (q, k, v, out, lse, dout))
    bo, bq, bk, bv = (np.zeros(q.shape) for _ in range(4))
    for h in range(q.shape[1]):
        mask = ob.visible(cu, idx, cnt, h)
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(mask, np.exp(scale * (q[:, h] @ k[:, h].T) - lse[:, h, None]), 0.0)
        av, ado, ao = np.abs(v[:, h]), np.abs(dout[:, h]), np.abs(out[:, h])
        bo[:, h] = (HALF + EXP) * (p @ av + ao)
        bv[:, h] = (HALF + EXP) * (p.T @ ado)
        delta = (dout[:, h] * out[:, h]).sum(1, keepdims=True)
        ds = np.abs(scale * p * (dout[:, h] @ v[:, h].T - delta))
        e = HALF * ds + EXP * abs(scale) * p * (ado @ av.T + (ado * ao).sum(1, keepdims=True)) + 2 * EXP * ds
        bq[:, h], bk[:, h] = e @ np.abs(k[:, h]), e.T @ np.abs(q[:, h])
    return bo, bq, bk, bv


def _within(got, ref, bound, what):
    got = got.double().cpu().numpy()
    err, lim = np.abs(got - ref), bound + HALF * (1 + HALF) * np.abs(ref) + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= lim).all(), f"{what}: worst {float((err / lim).max()):.2f} of the bound"


def _check(dev, lens, H, d, idx, cnt, seed=1, scale=None, data=None, max_seqlen=None):
    q, k, v, dout, cu, longest = _inputs(lens, H, d, seed) if data is None else data
    scale = d ** -0.5 if scale is None else scale
    longest = longest if max_seqlen is None else max_seqlen
    g = [t.to(dev) for t in (q, k, v, dout, cu)]
    gi = torch.as_tensor(idx).to(dev).contiguous()
    gc = torch.as_tensor(cnt).to(dev).contiguous()
    out, lse = pa.block_sparse_attn_fwd(g[0], g[1], g[2], g[4], longest, gi, gc, scale)
    dq, dk, dv = pa.block_sparse_attn_bwd(g[0], g[1], g[2], out, lse, g[3], g[4], longest, gi, gc, scale)
    assert pa.pa_get_error() == pa.PA_OK
    idx, cnt, cu = gi.cpu().numpy(), gc.cpu().numpy(), cu.numpy()
    ro, rl = ob.sparse_attention(q, k, v, cu, idx, cnt, scale)
    rg = ob.sparse_attention_bwd(q, k, v, out, lse, dout, cu, idx, cnt, scale)
    bo, bq, bk, bv = _bounds(q, k, v, ro, rl, dout, cu, idx, cnt, scale)
    _within(out, ro, bo, "out")
    got_l = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got_l), np.isneginf(rl))
    some = np.isfinite(rl)
    assert np.abs(got_l[some] - rl[some]).max(initial=0.0) <= 2e-4
    for name, a, b, lim in zip(("dq", "dk", "dv"), (dq, dk, dv), rg, (bq, bk, bv)):
        _within(a, b, lim, name)
    return out, lse, dq, dk, dv


def _random_lists(lens, H, width, seed, empty=0.15):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)])
    rows = ob.table_rows(len(lens), int(cu[-1]))
    # unread entries hold numbers that would be out of range
    idx = rng.integers(-2 ** 31, 2 ** 31 - 1, (H, rows, width)).astype(np.int32)
    cnt = rng.integers(-2 ** 31, 2 ** 31 - 1, (H, rows)).astype(np.int32)
    for s, n in enumerate(lens):
        nb = ob.n_blocks(n)
        for b in range(nb):
            for h in range(H):
                m = 0 if rng.random() < empty else int(rng.integers(1, min(nb, width) + 1))
                idx[h, ob.first_row(cu, s) + b, :m] = np.sort(rng.choice(nb, m, replace=False))
                cnt[h, ob.first_row(cu, s) + b] = m
    return idx, cnt


PACKS = [[1], [128], [129], [257, 0, 5], [300, 64, 1000], [1, 127, 128, 129, 255, 256, 257, 384, 511], [0, 0, 700]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", PACKS)
@pytest.mark.parametrize("density,floor", [(0.0, 1), (0.3, 2), (1.0, 1)])
def test_select_is_the_oracles(cuda_device, lens, d, density, floor):
    H = 3
    q, k, *_ , cu, longest = _inputs(lens, H, d, 20)
    idx, cnt = pa.block_select(q.to(cuda_device), k.to(cuda_device), cu.to(cuda_device), longest, density, floor)
    assert pa.pa_get_error() == pa.PA_OK
    ri, rc = ob.block_select(q, k, cu.numpy(), density, floor, idx.shape[2])
    assert np.array_equal(cnt.cpu().numpy(), rc) and np.array_equal(idx.cpu().numpy(), ri)


def test_select_ties_nan_and_infinity(cuda_device):
    lens, H, d = [1100, 200], 2, 64
    q, k, _, _, cu, longest = _inputs(lens, H, d, 21)
    q[:256] = 0  # every score of these blocks is 0: the lowest blocks
    k[300] = float("nan")
    k[600, 0] = float("inf")
    k[700, 0] = float("-inf")
    for floor in (1, 4, 8, 9):
        idx, cnt = pa.block_select(q.to(cuda_device), k.to(cuda_device), cu.to(cuda_device), longest, 0.0, floor)
        with np.errstate(invalid="ignore"):
            ri, rc = ob.block_select(q, k, cu.numpy(), 0.0, floor, idx.shape[2])
        assert np.array_equal(cnt.cpu().numpy(), rc) and np.array_equal(idx.cpu().numpy(), ri)


@pytest.mark.parametrize("lq,lk", [(-131, 0), (0, -131), (119, -100), (-60, 60), (119, 119)])
def test_select_over_the_types_whole_range(cuda_device, lq, lk):
    """Subnormal values and the largest: products down to 2^-260 and up to 2^254, which 64 bits hold exactly scaled."""
    lens, H, d = [1500, 130], 3, 128
    q, k, _, _, cu, longest = _inputs(lens, H, d, 23)
    q, k = (torch.from_numpy(np.ldexp(x.double().numpy(), e)).to(torch.bfloat16) for x, e in ((q, lq), (k, lk)))
    assert torch.isfinite(q).all() and torch.isfinite(k).all() and (q != 0).any() and (k != 0).any()
    idx, cnt = pa.block_select(q.to(cuda_device), k.to(cuda_device), cu.to(cuda_device), longest, 0.4, 1)
    ri, rc = ob.block_select(q, k, cu.numpy(), 0.4, 1, idx.shape[2])
    assert np.array_equal(cnt.cpu().numpy(), rc) and np.array_equal(idx.cpu().numpy(), ri)


def test_select_many_blocks_and_wider_tables(cuda_device):
    """A segment of 300 blocks (several words of each structure), max_seqlen above the longest, 40 short images."""
    for lens, H, d, density in (([128 * 300 - 5], 2, 64, 0.1), ([40] * 40 + [2000], 25, 64, 0.5)):
        q, k, _, _, cu, longest = _inputs(lens, H, d, 22)
        idx, cnt = pa.block_select(q.to(cuda_device), k.to(cuda_device), cu.to(cuda_device), longest + 1000, density, 3)
        ri, rc = ob.block_select(q, k, cu.numpy(), density, 3, idx.shape[2])
        assert np.array_equal(cnt.cpu().numpy(), rc) and np.array_equal(idx.cpu().numpy(), ri)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", PACKS)
def test_selected_blocks(cuda_device, lens, d):
    H = 2
    data = _inputs(lens, H, d, 23)
    idx, cnt = ob.block_select(data[0], data[1], data[4].numpy(), 0.4, 1, max(1, ob.keep_count(max(lens), 0.4, 1)))
    _check(cuda_device, lens, H, d, idx, cnt, data=data)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H,width", [([700], 3, 6), ([300, 1500], 2, 5), ([90] * 12, 2, 1), ([1280, 0, 33], 4, 10)])
def test_callers_own_lists(cuda_device, lens, H, width, d):
    """Lists of any length with empty rows, keys that nobody sees, and unread table entries that hold anything."""
    idx, cnt = _random_lists(lens, H, width, 24)
    _check(cuda_device, lens, H, d, idx, cnt, seed=25)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.6])
def test_scales(cuda_device, scale):
    idx, cnt = _random_lists([500, 260], 2, 4, 26)
    _check(cuda_device, [500, 260], 2, 64, idx, cnt, seed=27, scale=scale)
    _check(cuda_device, [500, 260], 2, 128, idx, cnt, seed=28, scale=scale)


def test_sorted_work_and_a_loose_max_seqlen(cuda_device):
    """More items than CTAs (the longest-first path) with lists of very different lengths."""
    lens, H = [1500, 60, 60, 700], 40
    idx, cnt = _random_lists(lens, H, 12, 29)
    _check(cuda_device, lens, H, 64, idx, cnt, seed=30, max_seqlen=100000)


def test_all_empty(cuda_device):
    lens, H = [300], 2
    cu = np.array([0, 300])
    idx = np.zeros((H, ob.table_rows(1, 300), 2), dtype=np.int32)
    cnt = np.zeros((H, ob.table_rows(1, 300)), dtype=np.int32)
    out, lse, dq, dk, dv = _check(cuda_device, lens, H, 64, idx, cnt)
    for t in (out, dq, dk, dv):
        assert not t.any()
    assert torch.isneginf(lse).all() and cu[-1] == 300


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_listed_does_not_leak(cuda_device, d, bad):
    """A NaN or infinity in a block that no list names, or in the next image (behind a short last block), changes no bit."""
    lens, H = [330, 200], 2
    q, k, v, dout, cu, longest = _inputs(lens, H, d, 31)
    rows = ob.table_rows(2, 530)
    idx = np.zeros((H, rows, 2), dtype=np.int32)
    cnt = np.zeros((H, rows), dtype=np.int32)
    idx[:, 0:3] = [0, 2]  # nobody names block 1 of the first image
    cnt[:, 0:3] = 2
    r1 = ob.first_row(cu.numpy(), 1)
    idx[:, r1:r1 + 2, 0] = [[0], [1]][0]
    cnt[:, r1:r1 + 2] = 1
    gi, gc = torch.from_numpy(idx).to(cuda_device), torch.from_numpy(cnt).to(cuda_device)

    def run(q, k, v, dout):
        g = [t.to(cuda_device) for t in (q, k, v, dout, cu)]
        out, lse = pa.block_sparse_attn_fwd(g[0], g[1], g[2], g[4], longest, gi, gc)
        # dq is summed in no fixed order: compare what is deterministic bit for bit, dq to a rounding
        return (out, lse) + pa.block_sparse_attn_bwd(g[0], g[1], g[2], out, lse, g[3], g[4], longest, gi, gc)

    want = run(q, k, v, dout)
    k2, v2 = k.clone(), v.clone()
    k2[130:200], v2[130:200] = bad, bad
    q3, d3 = q.clone(), dout.clone()
    for t in (k2, v2, q3, d3):
        t[330:] = bad  # the second image, whole
    got = run(q3, k2, v2, d3)
    for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, want):
        a, b = a[:330], b[:330]
        assert torch.isfinite(a.float()).all(), name
        if name == "dq":
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-6)
        else:
            assert torch.equal(a, b), name


def test_everything_listed_is_the_dense_attention(cuda_device):
    lens, H, d = [640, 200, 1], 3, 128
    q, k, v, dout, cu, longest = (t.to(cuda_device) if torch.is_tensor(t) else t for t in _inputs(lens, H, d, 32))
    idx, cnt = pa.block_select(q, k, cu, longest, 1.0)
    out, lse = pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt)
    ro, rl = pa.varlen_attn_fwd(q, k, v, cu, longest)
    assert torch.allclose(out.float(), ro.float(), rtol=2.0 ** -7, atol=2e-3) and torch.allclose(lse, rl, atol=1e-4)
    for a, b in zip(pa.block_sparse_attn_bwd(q, k, v, out, lse, dout, cu, longest, idx, cnt),
                    pa.varlen_attn_bwd(q, k, v, ro, rl, dout, cu, longest)):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -7 * float(b.float().abs().max()))


def test_repeatable(cuda_device):
    lens, H, d = [900, 300], 6, 64
    q, k, v, dout, cu, longest = (t.to(cuda_device) if torch.is_tensor(t) else t for t in _inputs(lens, H, d, 33))
    idx, cnt = pa.block_select(q, k, cu, longest, 0.5)
    a = pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt)
    g = pa.block_sparse_attn_bwd(q, k, v, *a, dout, cu, longest, idx, cnt)
    for _ in range(3):
        b = pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        g2 = pa.block_sparse_attn_bwd(q, k, v, *a, dout, cu, longest, idx, cnt)
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
        assert torch.allclose(g[0].float(), g2[0].float(), rtol=2.0 ** -7, atol=1e-6)


def test_bad_lists_and_packs_are_recorded(cuda_device):
    lens, H, d = [300, 200], 2, 64
    q, k, v, dout, cu, longest = (t.to(cuda_device) if torch.is_tensor(t) else t for t in _inputs(lens, H, d, 34))
    idx, cnt = pa.block_select(q, k, cu, longest, 1.0)
    out, lse = pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt)
    assert pa.pa_get_error() == pa.PA_OK

    def both(code, cu=cu, longest=longest, idx=idx, cnt=cnt):
        pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt)
        assert pa.pa_get_error() == code
        pa.block_sparse_attn_bwd(q, k, v, out, lse, dout, cu, longest, idx, cnt)
        assert pa.pa_get_error() == code

    both(pa.PA_OK)
    for at, value in (((0, 0, 0), 1), ((1, 2, 2), 3), ((0, 1, 0), -1), ((0, 1, 1), 2 ** 30), ((1, 0, 1), 0)):
        wrong = idx.clone()
        wrong[at] = value  # (0, 0, 0) <- 1 repeats block 1
        both(pa.PA_ERR_BLOCKS, idx=wrong)
    for value in (-1, idx.shape[2] + 1, 2 ** 31 - 1):
        wrong = cnt.clone()
        wrong[0, 1] = value
        both(pa.PA_ERR_BLOCKS, cnt=wrong)
    both(pa.PA_ERR_MAX_SEQLEN, longest=299)
    for bad in ([0, 300, 499], [0, 520, 500], [-1, 300, 500]):
        wrong = torch.tensor(bad, dtype=torch.int32, device=cuda_device)
        both(pa.PA_ERR_CU_SEQLENS, cu=wrong)
        pa.block_select(q, k, wrong, 300, 1.0)
        assert pa.pa_get_error() == pa.PA_ERR_CU_SEQLENS
    pa.block_select(q, k, cu, 299, 1.0)
    assert pa.pa_get_error() == pa.PA_ERR_MAX_SEQLEN
    both(pa.PA_OK)


@pytest.mark.parametrize("bad", [[0, 5000, 300, 6000], [0, 3000, 2000, 2500, 1000, 6000], [0, 6000, 0, 6000], [0, 0, -5, 6000]])
def test_packs_that_decrease_are_recorded(cuda_device, bad):
    """Segments that overlap, of which some blocks' rows are found to be another segment's; into fresh workspaces."""
    H, d = 2, 64
    q, k, v, dout, cu, longest = (t.to(cuda_device) if torch.is_tensor(t) else t for t in _inputs([6000], H, d, 36))
    rows = ob.table_rows(len(bad) - 1, 6000)
    idx = torch.arange(3, dtype=torch.int32, device=cuda_device).repeat(H, rows, 1)
    cnt = torch.full((H, rows), 3, dtype=torch.int32, device=cuda_device)
    wrong = torch.tensor(bad, dtype=torch.int32, device=cuda_device)
    out, lse = torch.zeros_like(q), torch.zeros((6000, H), device=cuda_device)
    for backward in (0, 1):
        n = pa.pa_block_sparse_workspace_bytes(len(bad) - 1, 6000, H, d, longest, 3, backward)
        ws = torch.zeros(n, dtype=torch.uint8, device=cuda_device)
        if backward:
            g = [torch.empty_like(q) for _ in range(3)]
            assert pa.pa_block_sparse_attn_bwd(q, k, v, out, lse, dout, wrong, longest, idx, cnt, 0.1, *g, ws) == pa.PA_OK
        else:
            assert pa.pa_block_sparse_attn_fwd(q, k, v, wrong, longest, idx, cnt, 0.1, out, lse, ws) == pa.PA_OK
        assert pa.pa_get_error() == pa.PA_ERR_CU_SEQLENS
    pa.block_select(q, k, wrong, longest, 0.3)
    assert pa.pa_get_error() == pa.PA_ERR_CU_SEQLENS


def test_no_tokens(cuda_device):
    cu = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    idx, cnt = pa.block_select(q, q, cu, 128, 1.0)
    assert (idx == -1).all() and not cnt.any() and cnt.shape == (2, 2)
    out, lse = pa.block_sparse_attn_fwd(q, q, q, cu, 128, idx, cnt)
    assert out.shape == q.shape and all(t.shape == q.shape for t in pa.block_sparse_attn_bwd(
        q, q, q, out, lse, q, cu, 128, idx, cnt))


def test_streams_and_graphs(cuda_device):
    """A fresh stream, and two captured graphs (one on a stream the library has not seen) replayed at once."""
    lens, H, d = [700, 200], 30, 64
    q, k, v, dout, cu, longest = (t.to(cuda_device) if torch.is_tensor(t) else t for t in _inputs(lens, H, d, 35))

    def everything(stream=None):
        idx, cnt = pa.block_select(q, k, cu, longest, 0.5, stream=stream)
        out, lse = pa.block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt, stream=stream)
        return (idx, cnt, out, lse) + pa.block_sparse_attn_bwd(q, k, v, out, lse, dout, cu, longest, idx, cnt,
                                                               stream=stream)

    def same(got, want):
        for i, (a, b) in enumerate(zip(got, want)):
            if i == 4:  # dq
                assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-6)
            else:
                assert torch.equal(a, b), i

    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = everything(side)
    assert pa.pa_get_error(side) == pa.PA_OK
    same(got, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            res = everything()
        graphs.append((g, res))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, res), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                res[2].zero_()
                g.replay()
    torch.cuda.synchronize()
    for _, res in graphs:
        same(res, want)
    assert pa.pa_get_error() == pa.PA_OK
