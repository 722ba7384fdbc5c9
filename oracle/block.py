"""fp64 oracle for what stands around and inside the packed attention in a DiT block: the gated residual join with
its norms, the rotation by positions with several axes, the selection of key blocks and the attention over them,
and the gradients of each.

TEST INFRASTRUCTURE ONLY; it shares no code with the CUDA path.  Plain numpy in fp64, written from the definitions
of ``include/packattn_block.h``; gradients are the formulas' (pinned against differences in the tests).
"""
import math

import numpy as np

BLOCK = 128


def f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        return x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def segment_ids(cu, total):
    cu = np.asarray(cu, dtype=np.int64)
    return np.repeat(np.arange(len(cu) - 1), np.diff(cu))[:total]


# ---------------------------------------------------------------- norms, gate, residual

def normed(v, kind, eps):
    """(N(v), 1 / deviation) over the last axis; kind none, layer or rms."""
    if kind == "none":
        return v, np.ones(v.shape[:-1] + (1,))
    mu = v.mean(-1, keepdims=True) if kind == "layer" else 0.0
    rstd = 1.0 / np.sqrt(((v - mu) ** 2).mean(-1, keepdims=True) + eps)
    return (v - mu) * rstd, rstd


def _rows(m, seg, one, shape):
    return np.full(shape, one) if m is None else f64(m)[seg]


def _vec(w, c):
    return np.ones(c) if w is None else f64(w)


def join(x, cu, y, gate, post, w_post, res, eps=1e-6):
    """r before its rounding."""
    x, y = f64(x), f64(y)
    seg = segment_ids(cu, len(x))
    return res * x + _rows(gate, seg, 1.0, x.shape) * normed(y, post, eps)[0] * _vec(w_post, x.shape[1])


def front(r, cu, pre, w_pre, scale, shift, eps=1e-6):
    """z before its rounding, from the stored r."""
    r = f64(r)
    seg = segment_ids(cu, len(r))
    hat = normed(r, pre, eps)[0]
    return hat * _vec(w_pre, r.shape[1]) * (1.0 + _rows(scale, seg, 0.0, r.shape)) + _rows(shift, seg, 0.0, r.shape)


def norm_back(g, hat, rstd, kind):
    if kind == "none":
        return g
    g = g - hat * (g * hat).mean(-1, keepdims=True) - (g.mean(-1, keepdims=True) if kind == "layer" else 0.0)
    return g * rstd


def block_norm_bwd(r, cu, dr, dz, y=None, gate=None, post="none", w_post=None, res=1.0, pre="layer", w_pre=None,
                   scale=None, shift=None, eps=1e-6):
    """Gradients of the join; dict of fp64 arrays (dy None without y; the sums always)."""
    r, y = f64(r), f64(y)
    T, C = r.shape
    B = len(cu) - 1
    seg = segment_ids(cu, T)

    def by_segment(v):
        out = np.zeros((B, C))
        np.add.at(out, seg, v)
        return out

    total = np.zeros((T, C)) if dr is None else f64(dr)
    out = {}
    if dz is not None:
        dz = f64(dz)
        hat, rstd = normed(r, pre, eps)
        w, up = _vec(w_pre, C), 1.0 + _rows(scale, seg, 0.0, r.shape)
        out["dscale"], out["dshift"] = by_segment(dz * hat * w), by_segment(dz)
        out["dw_pre"] = (dz * up * hat).sum(0)
        total = total + norm_back(dz * up * w, hat, rstd, pre)
    out["dx"], out["dr"] = res * total, total
    if y is not None:
        hat, rstd = normed(y, post, eps)
        w, g = _vec(w_post, C), _rows(gate, seg, 1.0, r.shape)
        out["dgate"] = by_segment(total * hat * w)
        out["dw_post"] = (total * g * hat).sum(0)
        out["dy"] = norm_back(total * g * w, hat, rstd, post)
    return out


# ---------------------------------------------------------------- rotary positions with several axes

def rope_axes(x, pos, dims, theta, interleaved=False, inverse=False):
    """x [T, H, d] rotated; theta one base or one per axis."""
    x, pos = f64(x).copy(), f64(pos)
    d = x.shape[-1]
    bases = [theta] * len(dims) if np.isscalar(theta) else list(theta)
    p = 0
    for a, n in enumerate(dims):
        for i in range(n // 2):
            ang = pos[:, a] * bases[a] ** (-2.0 * i / n) * (-1.0 if inverse else 1.0)
            c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
            lo, hi = (2 * p, 2 * p + 1) if interleaved else (p, p + d // 2)
            u, v = x[..., lo].copy(), x[..., hi].copy()
            x[..., lo], x[..., hi] = u * c - v * s, u * s + v * c
            p += 1
    return x


# ---------------------------------------------------------------- attention over selected blocks

def n_blocks(length):
    return (int(length) + BLOCK - 1) // BLOCK


def keep_count(length, density, min_blocks):
    nb = n_blocks(length)
    return min(nb, max(min_blocks, math.ceil(density * nb)))


def first_row(cu, s):
    return int(cu[s]) // BLOCK + s


def table_rows(batch, total):
    return total // BLOCK + batch


def block_select(q, k, cu, density, min_blocks, width):
    """(idx int32 [H, rows, width], cnt int32 [H, rows])."""
    q, k = f64(q), f64(k)
    T, H, _ = q.shape
    B = len(cu) - 1
    idx = np.full((H, table_rows(B, T), width), -1, dtype=np.int32)
    cnt = np.zeros((H, table_rows(B, T)), dtype=np.int32)
    for s in range(B):
        a, b = int(cu[s]), int(cu[s + 1])
        nb = n_blocks(b - a)
        if nb == 0:
            continue
        mean = [np.stack([x[a + i * BLOCK:min(a + (i + 1) * BLOCK, b)].mean(0) for i in range(nb)]) for x in (q, k)]
        score = np.einsum("ihd,jhd->hij", *mean)
        score = np.where(np.isnan(score), -np.inf, score)
        keep = keep_count(b - a, density, min_blocks)
        order = np.argsort(-score, axis=-1, kind="stable")[..., :keep]
        rows = slice(first_row(cu, s), first_row(cu, s) + nb)
        idx[:, rows, :keep] = np.sort(order, axis=-1)
        cnt[:, rows] = keep
    return idx, cnt


def visible(cu, idx, cnt, head):
    """[T, T] bool: which keys a query row of this head sees."""
    T = int(cu[-1])
    out = np.zeros((T, T), dtype=bool)
    for s in range(len(cu) - 1):
        a, b = int(cu[s]), int(cu[s + 1])
        for i in range(n_blocks(b - a)):
            row = first_row(cu, s) + i
            for j in np.asarray(idx[head, row, :int(cnt[head, row])]):
                out[a + i * BLOCK:min(a + (i + 1) * BLOCK, b), a + j * BLOCK:min(a + (j + 1) * BLOCK, b)] = True
    return out


def sparse_attention(q, k, v, cu, idx, cnt, scale):
    """(out, lse); a row that sees no key has out = 0 and lse = -inf."""
    q, k, v = f64(q), f64(k), f64(v)
    T, H, d = q.shape
    out, lse = np.zeros((T, H, d)), np.full((T, H), -np.inf)
    for h in range(H):
        mask = visible(cu, idx, cnt, h)
        some = mask.any(1)
        s = np.where(mask, scale * (q[:, h] @ k[:, h].T), -np.inf)[some]
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        t = e.sum(1, keepdims=True)
        out[some, h] = e @ v[:, h] / t
        lse[some, h] = (m + np.log(t))[:, 0]
    return out, lse


def sparse_attention_bwd(q, k, v, out, lse, dout, cu, idx, cnt, scale):
    """(dq, dk, dv) with the given out and lse."""
    q, k, v, out, lse, dout = (f64(t) for t in (q, k, v, out, lse, dout))
    dq, dk, dv = (np.zeros(q.shape) for _ in range(3))
    for h in range(q.shape[1]):
        mask = visible(cu, idx, cnt, h)
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(mask, np.exp(scale * (q[:, h] @ k[:, h].T) - lse[:, h, None]), 0.0)
        delta = (dout[:, h] * out[:, h]).sum(1, keepdims=True)
        ds = scale * p * (dout[:, h] @ v[:, h].T - delta)
        dq[:, h], dk[:, h], dv[:, h] = ds @ k[:, h], ds.T @ q[:, h], p.T @ dout[:, h]
    return dq, dk, dv
