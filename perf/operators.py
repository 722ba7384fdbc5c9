"""The operators around and inside a packed DiT block, as cases that can be timed.

Five operators, all over a pack of images (``cu_seqlens`` splits the token stream):

* ``norm``      gated residual join with the norm behind a block and the norm in front of the next;
* ``norm_bwd``  its gradients;
* ``rope``      rotary positions with several axes (time, height, width) on q and k, forward, backward, or
                inside the fused QKV projection;
* ``sparse``    attention over the key blocks that a cheap score selects for every block of queries;
* ``sparse_bwd``  its gradients.

``run`` computes them in plain torch operations, or through the package where ``own`` is true.
"""
import math
import random

import torch

own = False

BLOCK = 128  # tokens of a query block and of a key block
DEVICE = "cuda"
EPS = 1e-6

# packs of this repository's workloads: image sizes at patch 16
TINY = "256,108"
MIXED = "1024,4096,1296"
TRAINING = "2088,2592,2397,3600,3538,3060,272,2035,2028,1782,3150,2132,2106,3648,3480,2900"


def listed():
    return [
        # a pair of small images through the norm in front of the first block: latency counts
        dict(name="norm_tiny", op="norm", segments=TINY, hidden=128, f32=False, join=False, post="none", pre="layer",
             w=False, mod=True, res=1.0),
        # a mixed-resolution pack between two blocks: RMS norm behind, gate, residual, modulated layer norm in front
        dict(name="norm_mixed", op="norm", segments=MIXED, hidden=2048, f32=False, join=True, post="rms", pre="layer",
             w=True, mod=True, res=1.0),
        # a training pack with the residual stream in 32 bits and a scaled residual
        dict(name="norm_training", op="norm", segments=TRAINING, hidden=1536, f32=True, join=True, post="none",
             pre="rms", w=True, mod=True, res=0.70710678),
        # the gradients of the mixed pack's join
        dict(name="norm_bwd_mixed", op="norm_bwd", segments=MIXED, hidden=2048, f32=False, join=True, post="rms",
             pre="layer", w=True, mod=True, res=1.0),
        # thousands of thumbnails: as many rows of modulation gradients as images
        dict(name="norm_bwd_thumbs", op="norm_bwd", segments="thumbs:2048:5", hidden=1152, f32=True, join=True,
             post="none", pre="layer", w=False, mod=True, res=1.0),
        # q and k of the mixed pack, image positions (frame, row, column)
        dict(name="rope_mixed", op="rope", segments=MIXED, heads=24, head_dim=128, dims="16,56,56", theta=10000.0,
             inter=False, bwd=False, hidden=0),
        # the gradients of a long video's q and k, interleaved pairs
        dict(name="rope_bwd_long", op="rope", segments="65536", heads=8, head_dim=64, dims="16,24,24", theta=256.0,
             inter=True, bwd=True, hidden=0),
        # the projection of the mixed pack with the rotation in its epilogue
        dict(name="rope_qkv_mixed", op="rope", segments=MIXED, heads=16, head_dim=128, dims="16,56,56", theta=10000.0,
             inter=False, bwd=False, hidden=2048),
        # the smallest sparse call: two images, three blocks
        dict(name="sparse_tiny", op="sparse", segments=TINY, heads=2, head_dim=64, density=0.5, floor=1),
        # one 2048 x 2048 image in serving, an eighth of the blocks
        dict(name="sparse_interactive", op="sparse", segments="16384", heads=24, head_dim=128, density=0.125, floor=4),
        # training on the mixed pack with a quarter of the blocks
        dict(name="sparse_bwd_mixed", op="sparse_bwd", segments=MIXED, heads=24, head_dim=128, density=0.25, floor=4),
        # a long video in training, a sixteenth of the blocks
        dict(name="sparse_bwd_long", op="sparse_bwd", segments="65536", heads=8, head_dim=64, density=0.0625, floor=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_segments(rng, total, most):
    """Image token counts that sum to at most `total`: one image, a few, or many; an empty one now and then."""
    n = min(_log(rng, 1, most), total)
    weights = [math.exp(rng.uniform(-1.5, 1.5)) for _ in range(n)]
    lens = [max(1, int(total * w / sum(weights))) for w in weights]
    if rng.random() < 0.2:
        lens.insert(rng.randrange(len(lens) + 1), 0)
    return ",".join(str(x) for x in lens)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "sparse", "sparse_bwd"])
    if op in ("norm", "norm_bwd"):
        c = 8 * _log(rng, 8, 512)
        total = _log(rng, 1, min(60000, int(4.5e7 / c)))
        join = rng.random() < 0.75
        pre = rng.choice(["layer", "rms"] + (["none"] if join else []))
        return dict(op=op, segments=_draw_segments(rng, total, 300), hidden=c, f32=rng.random() < 0.5, join=join,
                    post=rng.choice(["none", "rms", "layer"]) if join else "none", pre=pre, w=rng.random() < 0.5,
                    mod=rng.random() < 0.75, res=rng.choice([1.0, 0.5]) if join else 1.0)
    if op == "rope":
        d = rng.choice([64, 128])
        h = rng.randint(1, 24)
        dims = rng.choice({64: ["16,24,24", "32,32", "64", "8,16,16"], 128: ["16,56,56", "64,64", "128", "32,32,32,32",
                                                                             "16,24,24"]}[d])
        hidden = 8 * _log(rng, 8, 256) if rng.random() < 0.3 else 0
        total = _log(rng, 1, int((2.0e7 if not hidden else 1.0e7) / (h * d)))
        return dict(op=op, segments=_draw_segments(rng, total, 100), heads=h, head_dim=d, dims=dims,
                    theta=rng.choice([10000.0, 256.0]), inter=rng.random() < 0.5,
                    bwd=rng.random() < 0.5 and not hidden, hidden=hidden)
    d = rng.choice([64, 128])
    h = rng.randint(1, 24)
    total = _log(rng, 1, int(math.sqrt(1.0e9 / h)))
    return dict(op=op, segments=_draw_segments(rng, total, 40), heads=h, head_dim=d,
                density=rng.choice([0.0, 0.0625, 0.125, 0.25]) if total > 8192 else rng.choice([0.0, 0.125, 0.5, 1.0]),
                floor=rng.randint(1, 6))


# ---------------------------------------------------------------- inputs

def _segments(case):
    text = case["segments"]
    if text.startswith("thumbs:"):
        _, n, seed = text.split(":")
        rng = random.Random(int(seed))
        return [rng.randint(1, 11) * rng.randint(1, 11) for _ in range(int(n))]
    return [int(x) for x in text.split(",")]


def _blocks(length):
    return (length + BLOCK - 1) // BLOCK


def _keep(case, length):
    """Key blocks that every query block of a segment keeps."""
    nb = _blocks(length)
    return min(nb, max(case["floor"], math.ceil(case["density"] * nb)))


def _rows(lens):
    """First row of every segment in the table of query blocks, and the number of rows."""
    out, at = [], 0
    for s, n in enumerate(lens):
        out.append(at // BLOCK + s)
        at += n
    return out, at // BLOCK + len(lens)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _positions(lens):
    """(frame, row, column, token) of every token: images of about square shape, 16 rows a frame on long ones."""
    out = []
    for n in lens:
        i = torch.arange(n, device=DEVICE)
        wid = max(1, int(math.ceil(math.sqrt(n))))
        hei = wid if n <= 4096 else max(1, wid // 4)
        out.append(torch.stack([i // (wid * hei), i // wid % hei, i % wid, i], dim=1))
    return torch.cat(out).float()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    lens = _segments(case)
    total = sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st = dict(case=case, lens=lens, longest=max(lens), cu=torch.tensor(cu, dtype=torch.int32, device=DEVICE))
    if case["op"] in ("norm", "norm_bwd"):
        c, wide = case["hidden"], torch.float32 if case["f32"] else torch.bfloat16
        # a residual stream with a few channels far larger than the rest
        channel = torch.exp(0.5 * _randn(g, c))
        channel[torch.randint(0, c, (max(1, c // 512),), generator=g, device=DEVICE)] *= 20.0
        mod = _randn(g, len(lens), 3, c, dtype=wide) * 0.3  # gate, scale, shift: slices of one projection's output
        st["x"] = ((_randn(g, total, c) + 0.1) * channel).to(wide)
        st["y"] = _randn(g, total, c, dtype=torch.bfloat16) if case["join"] else None
        st["gate"] = mod[:, 0] if case["mod"] and case["join"] else None
        st["scale"], st["shift"] = (mod[:, 1], mod[:, 2]) if case["mod"] and case["pre"] != "none" else (None, None)
        weights = [(1.0 + 0.2 * _randn(g, c)).to(wide) for _ in range(2)]
        st["w_post"] = weights[0] if case["w"] and case["post"] != "none" else None
        st["w_pre"] = weights[1] if case["w"] and case["pre"] != "none" else None
        if case["op"] == "norm_bwd":
            st["dr"] = _randn(g, total, c, dtype=wide) if case["join"] else None
            st["dz"] = _randn(g, total, c, dtype=torch.bfloat16) if case["pre"] != "none" else None
        return st
    h, d = case["heads"], case["head_dim"]
    if case["op"] == "rope":
        st["dims"] = [int(x) for x in case["dims"].split(",")]
        pos = _positions(lens)
        st["pos"] = (pos[:, 3:] if len(st["dims"]) == 1 else pos[:, :len(st["dims"])]).contiguous()
        if case["hidden"]:
            st["x"] = _randn(g, total, case["hidden"], dtype=torch.bfloat16)
            st["w"] = (_randn(g, 3 * h * d, case["hidden"]) * case["hidden"] ** -0.5).to(torch.bfloat16)
        else:
            st["q"], st["k"] = (_randn(g, total, h, d, dtype=torch.bfloat16) for _ in range(2))
        return st
    # neighbouring tokens of an image look alike: a slow part per 64 tokens and a part per token
    n64 = total // 64 + 1
    q, k = (torch.repeat_interleave(_randn(g, n64, h, d), 64, dim=0)[:total] * 0.7 + _randn(g, total, h, d) * 0.7
            for _ in range(2))
    st["q"], st["k"] = q.to(torch.bfloat16), k.to(torch.bfloat16)
    st["v"] = _randn(g, total, h, d, dtype=torch.bfloat16)
    if case["op"] == "sparse_bwd":
        st["idx"], st["cnt"] = _plain_select(st)
        st["out"], st["lse"] = _plain_attend(st, st["idx"])
        st["dout"] = _randn(g, total, h, d, dtype=torch.bfloat16)
    return st


# ---------------------------------------------------------------- plain forms

def _segment_of(st, total):
    return torch.searchsorted(st["cu"][1:].long(), torch.arange(total, device=DEVICE), right=True)


def _normed(v, kind):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * rstd, rstd


def _norm_back(g, hat, rstd, kind):
    g = g - hat * (g * hat).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if kind == "layer" else 0.0)
    return g * rstd


def _plain_norm(st):
    case, x = st["case"], st["x"]
    seg = _segment_of(st, x.shape[0])
    r, out = x, {}
    if st["y"] is not None:
        u = st["y"].float()
        if case["post"] != "none":
            u = _normed(u, case["post"])[0]
        if st["w_post"] is not None:
            u = u * st["w_post"].float()
        if st["gate"] is not None:
            u = u * st["gate"].float()[seg]
        r = (case["res"] * x.float() + u).to(x.dtype)
        out["r"] = r
    if case["pre"] != "none":
        z = _normed(r.float(), case["pre"])[0]
        if st["w_pre"] is not None:
            z = z * st["w_pre"].float()
        if st["scale"] is not None:
            z = z * (1.0 + st["scale"].float()[seg]) + st["shift"].float()[seg]
        out["z"] = z.to(torch.bfloat16)
    return out


def _by_segment(st, seg, v):
    out = torch.zeros(len(st["lens"]), v.shape[1], dtype=torch.float64, device=DEVICE)
    return out.index_add_(0, seg, v.double())


def _plain_norm_bwd(st):
    case, r = st["case"], st["x"]
    seg = _segment_of(st, r.shape[0])
    out = {}
    dr = st["dr"].float() if st["dr"] is not None else torch.zeros_like(r, dtype=torch.float32)
    if st["dz"] is not None:
        dz = st["dz"].float()
        hat, rstd = _normed(r.float(), case["pre"])
        sums = _by_segment(st, seg, dz * hat)
        up = 1.0 + st["scale"].float() if st["scale"] is not None else None
        if st["scale"] is not None:
            out["dscale"] = (sums * st["w_pre"].double() if st["w_pre"] is not None else sums).float()
            out["dshift"] = _by_segment(st, seg, dz).float()
        if st["w_pre"] is not None:
            out["dw_pre"] = (sums * up.double() if up is not None else sums).sum(0).float()
        g = dz
        if up is not None:
            g = g * up[seg]
        if st["w_pre"] is not None:
            g = g * st["w_pre"].float()
        dr = dr + _norm_back(g, hat, rstd, case["pre"])
    out["dx"] = (case["res"] * dr).to(r.dtype)
    if st["y"] is not None:
        hat, rstd = st["y"].float(), None
        if case["post"] != "none":
            hat, rstd = _normed(hat, case["post"])
        if st["gate"] is not None or st["w_post"] is not None:
            sums = _by_segment(st, seg, dr * hat)
        if st["gate"] is not None:
            out["dgate"] = (sums * st["w_post"].double() if st["w_post"] is not None else sums).float()
        if st["w_post"] is not None:
            out["dw_post"] = (sums * st["gate"].double() if st["gate"] is not None else sums).sum(0).float()
        g = dr
        if st["gate"] is not None:
            g = g * st["gate"].float()[seg]
        if st["w_post"] is not None:
            g = g * st["w_post"].float()
        out["dy"] = (_norm_back(g, hat, rstd, case["post"]) if rstd is not None else g).to(torch.bfloat16)
    return out


def _plain_angles(st):
    parts = []
    for a, n in enumerate(st["dims"]):
        freq = st["case"]["theta"] ** (-torch.arange(0, n, 2, dtype=torch.float64, device=DEVICE) / n)
        parts.append(st["pos"][:, a, None].double() * freq)
    ang = torch.cat(parts, dim=1)
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]


def _plain_rotate(x, cos, sin, inter):
    x, n, half = x.float(), cos.shape[-1], x.shape[-1] // 2
    y = x.clone()
    if inter:
        a, b, at, bt = x[..., 0:2 * n:2], x[..., 1:2 * n:2], slice(0, 2 * n, 2), slice(1, 2 * n, 2)
    else:
        a, b, at, bt = x[..., :n], x[..., half:half + n], slice(0, n), slice(half, half + n)
    y[..., at] = a * cos - b * sin
    y[..., bt] = a * sin + b * cos
    return y.to(torch.bfloat16)


def _plain_rope(st):
    case = st["case"]
    cos, sin = _plain_angles(st)
    if case["hidden"]:
        qkv = (st["x"].float() @ st["w"].float().t()).view(-1, 3, case["heads"], case["head_dim"])
        return dict(q=_plain_rotate(qkv[:, 0], cos, sin, case["inter"]),
                    k=_plain_rotate(qkv[:, 1], cos, sin, case["inter"]), v=qkv[:, 2].to(torch.bfloat16))
    if case["bwd"]:
        sin = -sin
    return dict(q=_plain_rotate(st["q"], cos, sin, case["inter"]), k=_plain_rotate(st["k"], cos, sin, case["inter"]))


def _to_blocks(x, length):
    """[L, H, d] of one segment as [H, blocks, 128, d], zeros behind the last token."""
    nb = _blocks(length)
    pad = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nb * BLOCK - length))
    return pad.view(nb, BLOCK, x.shape[1], x.shape[2]).permute(2, 0, 1, 3)


def _plain_select(st):
    case, lens = st["case"], st["lens"]
    h = case["heads"]
    first, rows = _rows(lens)
    width = _keep(case, st["longest"])
    idx = torch.full((h, rows, width), -1, dtype=torch.int32, device=DEVICE)
    cnt = torch.zeros(h, rows, dtype=torch.int32, device=DEVICE)
    at = 0
    for s, n in enumerate(lens):
        if n:
            nb, keep = _blocks(n), _keep(case, n)
            per = torch.full((nb, 1), float(BLOCK), dtype=torch.float64, device=DEVICE)
            per[-1] = n - (nb - 1) * BLOCK
            qm = _to_blocks(st["q"][at:at + n], n).double().sum(2) / per
            km = _to_blocks(st["k"][at:at + n], n).double().sum(2) / per
            score = qm @ km.transpose(1, 2)
            best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :keep]
            idx[:, first[s]:first[s] + nb, :keep] = torch.sort(best, dim=-1)[0].int()
            cnt[:, first[s]:first[s] + nb] = keep
        at += n
    return idx, cnt


def _gathered(st, idx):
    """Segment by segment and head group by head group: (heads, tokens, selected blocks, keys inside the image)."""
    case, lens = st["case"], st["lens"]
    first, _ = _rows(lens)
    at = 0
    for s, n in enumerate(lens):
        if n:
            nb, keep = _blocks(n), _keep(case, n)
            some = max(1, int(4e8 // (nb * BLOCK * keep * BLOCK)))
            for h0 in range(0, case["heads"], some):
                hs = slice(h0, min(h0 + some, case["heads"]))
                sel = idx[hs, first[s]:first[s] + nb, :keep].long()
                inside = (sel[..., None] * BLOCK + torch.arange(BLOCK, device=DEVICE) < n).flatten(2)[:, :, None]
                yield hs, slice(at, at + n), n, sel, inside
        at += n


def _take(x, n, sel):
    blocks = _to_blocks(x, n).float()
    return blocks, blocks[torch.arange(sel.shape[0], device=DEVICE)[:, None, None], sel].flatten(2, 3)


def _back(blocks, n):
    return blocks.flatten(1, 2)[:, :n].transpose(0, 1)


def _plain_attend(st, idx):
    out = torch.empty_like(st["q"])
    lse = torch.empty(out.shape[:2], dtype=torch.float32, device=DEVICE)
    scale = out.shape[2] ** -0.5
    for hs, ts, n, sel, inside in _gathered(st, idx):
        q = _to_blocks(st["q"][ts, hs], n).float()
        _, k = _take(st["k"][ts, hs], n, sel)
        _, v = _take(st["v"][ts, hs], n, sel)
        s = (q @ k.transpose(2, 3) * scale).masked_fill_(~inside, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        out[ts, hs] = _back(p @ v / total, n).to(torch.bfloat16)
        lse[ts, hs] = _back(top + torch.log(total), n)[..., 0]
    return out, lse


def _plain_attend_bwd(st):
    dq, dk, dv = (torch.empty_like(st["q"]) for _ in range(3))
    scale = dq.shape[2] ** -0.5
    for hs, ts, n, sel, inside in _gathered(st, st["idx"]):
        q, out, dout = (_to_blocks(st[x][ts, hs], n).float() for x in ("q", "out", "dout"))
        lse = _to_blocks(st["lse"][ts, hs, None], n)
        kb, k = _take(st["k"][ts, hs], n, sel)
        _, v = _take(st["v"][ts, hs], n, sel)
        p = torch.exp((q @ k.transpose(2, 3) * scale).masked_fill_(~inside, -math.inf) - lse)
        ds = p * (dout @ v.transpose(2, 3) - (dout * out).sum(-1, keepdim=True)) * scale
        dq[ts, hs] = _back(ds @ k, n).to(torch.bfloat16)
        to = (torch.arange(sel.shape[0], device=DEVICE)[:, None, None] * kb.shape[1] + sel).flatten()
        for grad, a, b in ((dk, ds, q), (dv, p, dout)):
            part = (a.transpose(2, 3) @ b).view(to.numel(), BLOCK, -1)
            total = torch.zeros_like(kb).flatten(0, 1).index_add_(0, to, part)
            grad[ts, hs] = _back(total.view_as(kb), n).to(torch.bfloat16)
    return dict(dq=dq, dk=dk, dv=dv)


# ---------------------------------------------------------------- one pass

def _own(st):
    import dit_resolution_packed_b200 as pa
    case, cu = st["case"], st["cu"]
    if case["op"] in ("norm", "norm_bwd"):
        how = dict(y=st["y"], gate=st["gate"], post=case["post"], w_post=st["w_post"], residual_scale=case["res"],
                   pre=case["pre"], w_pre=st["w_pre"], scale=st["scale"], shift=st["shift"], eps=EPS)
        if case["op"] == "norm_bwd":
            return {k: v for k, v in pa.block_norm_bwd(st["x"], cu, st["dr"], st["dz"], **how).items() if v is not None}
        r, z = pa.block_norm_fwd(st["x"], cu, **how)
        out = dict(r=r) if case["join"] else {}
        return dict(out, z=z) if z is not None else out
    if case["op"] == "rope":
        how = dict(dims=st["dims"], theta=case["theta"], interleaved=case["inter"])
        if case["hidden"]:
            q, k, v = pa.qkv_rope_axes_fwd(st["x"], st["w"], st["pos"], case["heads"], case["head_dim"], **how)
            return dict(q=q, k=k, v=v)
        q, k = (pa.rope_axes_bwd if case["bwd"] else pa.rope_axes_fwd)(st["q"], st["k"], st["pos"], **how)
        return dict(q=q, k=k)
    if case["op"] == "sparse":
        idx, cnt = pa.block_select(st["q"], st["k"], cu, st["longest"], case["density"], case["floor"])
        out, lse = pa.block_sparse_attn_fwd(st["q"], st["k"], st["v"], cu, st["longest"], idx, cnt)
        return dict(idx=idx, cnt=cnt, out=out, lse=lse)
    dq, dk, dv = pa.block_sparse_attn_bwd(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"], cu,
                                          st["longest"], st["idx"], st["cnt"])
    return dict(dq=dq, dk=dk, dv=dv)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    if op == "rope":
        return _plain_rope(state)
    if op == "sparse":
        idx, cnt = _plain_select(state)
        out, lse = _plain_attend(state, idx)
        return dict(idx=idx, cnt=cnt, out=out, lse=lse)
    return _plain_attend_bwd(state)


def work(case):
    lens = _segments(case)
    t, b = sum(lens), len(lens)
    if case["op"] in ("norm", "norm_bwd"):
        c, wide = case["hidden"], 4 if case["f32"] else 2
        given = c * wide * (2 * case["w"] + b * 3 * case["mod"])
        front, back = case["pre"] != "none", case["join"]
        if case["op"] == "norm":
            moved = t * c * (wide * (1 + back) + 2 * back + 2 * front)
            return dict(bytes=moved + given, flops=20.0 * t * c)
        moved = t * c * (wide * (2 + back) + 4 * back + 2 * front)
        return dict(bytes=moved + given + 4.0 * c * (2 * case["w"] + b * 3 * case["mod"]), flops=40.0 * t * c)
    h, d = case["heads"], case["head_dim"]
    if case["op"] == "rope":
        where = 4.0 * t * len(case["dims"].split(","))
        if case["hidden"]:
            n = 3 * h * d
            return dict(bytes=where + 2.0 * (t * case["hidden"] + n * case["hidden"] + t * n),
                        flops=2.0 * t * n * case["hidden"])
        return dict(bytes=where + 8.0 * t * h * d, flops=6.0 * t * h * d)
    # the pairs of a segment at the least: every query block may have kept the short last block
    pairs = sum(n * (_keep(case, n) * BLOCK - (_blocks(n) * BLOCK - n)) for n in lens if n)
    table = 4.0 * h * sum(_blocks(n) * (_keep(case, n) + 1) for n in lens if n)
    if case["op"] == "sparse":
        return dict(bytes=8.0 * t * h * d + 4.0 * t * h + table, flops=4.0 * pairs * d * h)
    return dict(bytes=16.0 * t * h * d + 4.0 * t * h + table, flops=10.0 * pairs * d * h)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(st):
    case = st["case"]
    x, y = st["x"].double(), st["y"]
    f64 = {k: st[k].double() if st[k] is not None else None for k in ("gate", "scale", "shift", "w_post", "w_pre")}
    out = {}
    z_at = []
    r = x.clone()
    at = 0
    for s, n in enumerate(st["lens"]):
        rows = slice(at, at + n)
        at += n
        if y is not None:
            u = y[rows].double()
            if case["post"] == "layer":
                u = (u - u.mean(1, keepdim=True)) / (u.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
            elif case["post"] == "rms":
                u = u / (u.square().mean(1, keepdim=True) + EPS).sqrt()
            u = u if f64["w_post"] is None else u * f64["w_post"]
            r[rows] = case["res"] * x[rows] + (u if f64["gate"] is None else f64["gate"][s] * u)
        if case["pre"] != "none":
            v = r[rows].to(st["x"].dtype).double()  # the norm is that of the stored residual
            if case["pre"] == "layer":
                v = (v - v.mean(1, keepdim=True)) / (v.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
            else:
                v = v / (v.square().mean(1, keepdim=True) + EPS).sqrt()
            v = v if f64["w_pre"] is None else v * f64["w_pre"]
            z_at.append(v if f64["scale"] is None else v + v * f64["scale"][s] + f64["shift"][s])
    if y is not None:
        out["r"] = r
    if z_at:
        out["z"] = torch.cat(z_at)
    return out


def _exact_norm_bwd(st):
    case = st["case"]
    leaf = {k: (st[k].double().requires_grad_() if st[k] is not None else None)
            for k in ("x", "y", "gate", "scale", "shift", "w_post", "w_pre")}
    seg = torch.repeat_interleave(torch.arange(len(st["lens"]), device=DEVICE), torch.tensor(st["lens"], device=DEVICE))

    def normed(v, kind):
        if kind == "layer":
            return (v - v.mean(1, keepdim=True)) / (v.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
        return v / (v.square().mean(1, keepdim=True) + EPS).sqrt() if kind == "rms" else v

    # first the gradient of the stored residual, then what the join passes on of it
    dr = st["dr"].double() if st["dr"] is not None else torch.zeros_like(leaf["x"])
    out = {}
    if st["dz"] is not None:
        z = normed(leaf["x"], case["pre"])
        z = z if leaf["w_pre"] is None else z * leaf["w_pre"]
        if leaf["scale"] is not None:
            z = z * (1.0 + leaf["scale"][seg]) + leaf["shift"][seg]
        z.backward(st["dz"].double())
        dr = dr + leaf["x"].grad
        if leaf["scale"] is not None:
            out["dscale"], out["dshift"] = leaf["scale"].grad, leaf["shift"].grad
        if leaf["w_pre"] is not None:
            out["dw_pre"] = leaf["w_pre"].grad
    out["dx"] = case["res"] * dr
    if leaf["y"] is not None:
        u = normed(leaf["y"], case["post"])
        u = u if leaf["w_post"] is None else u * leaf["w_post"]
        u = u if leaf["gate"] is None else u * leaf["gate"][seg]
        u.backward(dr)
        out["dy"] = leaf["y"].grad
        if leaf["gate"] is not None:
            out["dgate"] = leaf["gate"].grad
        if leaf["w_post"] is not None:
            out["dw_post"] = leaf["w_post"].grad
    return out


def _exact_rope(st):
    case = st["case"]
    parts = []
    for a, n in enumerate(st["dims"]):
        i = torch.arange(n // 2, device=DEVICE, dtype=torch.float64)
        parts.append(torch.outer(st["pos"][:, a].double(), torch.exp(-2.0 * i / n * math.log(case["theta"]))))
    angle = torch.cat(parts, 1)
    turn = torch.polar(torch.ones_like(angle), -angle if case["bwd"] else angle)[:, None]
    half, n = case["head_dim"] // 2, angle.shape[1]

    def rotated(x):
        pairs = x.unflatten(-1, (half, 2)) if case["inter"] else x.unflatten(-1, (2, half)).transpose(-1, -2)
        c = torch.view_as_complex(pairs.contiguous())
        c = torch.cat([c[..., :n] * turn, c[..., n:]], -1)
        pairs = torch.view_as_real(c)
        return (pairs if case["inter"] else pairs.transpose(-1, -2)).flatten(-2)

    if not case["hidden"]:
        return dict(q=rotated(st["q"].double()), k=rotated(st["k"].double()))
    y = torch.einsum("tc,nc->tn", st["x"].double(), st["w"].double())
    q, k, v = (p.unflatten(1, (case["heads"], case["head_dim"])) for p in y.chunk(3, dim=1))
    return dict(q=rotated(q), k=rotated(k), v=v)


def _exact_select(st):
    case, lens = st["case"], st["lens"]
    first, rows = _rows(lens)
    idx = torch.full((case["heads"], rows, _keep(case, st["longest"])), -1, dtype=torch.int32, device=DEVICE)
    cnt = torch.zeros(case["heads"], rows, dtype=torch.int32, device=DEVICE)
    at = 0
    for s, n in enumerate(lens):
        if not n:
            continue
        block = torch.arange(n, device=DEVICE) // BLOCK
        mean = {}
        for name in ("q", "k"):
            x = st[name][at:at + n].double()
            acc = torch.zeros(_blocks(n), *x.shape[1:], dtype=torch.float64, device=DEVICE).index_add_(0, block, x)
            mean[name] = acc / torch.bincount(block).double()[:, None, None]
        score = torch.einsum("ihd,jhd->hij", mean["q"], mean["k"])
        order = torch.argsort(-score, dim=-1, stable=True)
        keep = _keep(case, n)
        chosen = torch.zeros_like(score, dtype=torch.bool).scatter_(-1, order[..., :keep], True)
        idx[:, first[s]:first[s] + _blocks(n), :keep] = chosen.nonzero()[:, 2].view(*score.shape[:2], keep).int()
        cnt[:, first[s]:first[s] + _blocks(n)] = keep
        at += n
    return idx, cnt


def _exact_rows(st, idx):
    """(head, rows of queries, keys of the image, which keys each row sees) over the whole pack."""
    lens = st["lens"]
    first, _ = _rows(lens)
    at = 0
    for s, n in enumerate(lens):
        for h in range(st["case"]["heads"] if n else 0):
            sees = torch.zeros(_blocks(n), _blocks(n) + 1, dtype=torch.bool, device=DEVICE)
            sel = idx[h, first[s]:first[s] + _blocks(n)].long()
            sees.scatter_(1, torch.where(sel < 0, _blocks(n), sel), True)
            by_key = sees[:, :-1].repeat_interleave(BLOCK, 1)[:, :n]
            step = 16 * BLOCK
            for a in range(0, n, step):
                b = min(a + step, n)
                rows = by_key[a // BLOCK:_blocks(b)].repeat_interleave(BLOCK, 0)[:b - a]
                yield h, slice(at + a, at + b), slice(at, at + n), rows
        at += n


def _exact_sparse(st):
    idx, cnt = _exact_select(st)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device=DEVICE)
    for h, rows, keys, sees in _exact_rows(st, idx):
        s = st["q"][rows, h].double() @ st["k"][keys, h].double().T / math.sqrt(out.shape[2])
        s = torch.where(sees, s, -math.inf)
        lse[rows, h] = torch.logsumexp(s, 1)
        out[rows, h] = torch.softmax(s, 1) @ st["v"][keys, h].double()
    return dict(idx=idx, cnt=cnt, out=out, lse=lse)


def _exact_sparse_bwd(st):
    dq, dk, dv = (torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE) for _ in range(3))
    scale = 1.0 / math.sqrt(dq.shape[2])
    for h, rows, keys, sees in _exact_rows(st, st["idx"]):
        q, do = st["q"][rows, h].double(), st["dout"][rows, h].double()
        k, v = st["k"][keys, h].double(), st["v"][keys, h].double()
        p = torch.where(sees, torch.exp(scale * (q @ k.T) - st["lse"][rows, h].double()[:, None]), 0.0)
        mean = (do * st["out"][rows, h].double()).sum(1, keepdim=True)
        ds = scale * p * (do @ v.T - mean)
        dv[keys, h] += p.T @ do
        dk[keys, h] += ds.T @ q
        dq[rows, h] = ds @ k
    return dict(dq=dq, dk=dk, dv=dv)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(norm=_exact_norm, norm_bwd=_exact_norm_bwd, rope=_exact_rope, sparse=_exact_sparse,
                sparse_bwd=_exact_sparse_bwd)[case["op"]](st)
