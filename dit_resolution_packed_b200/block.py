"""Binding of ``include/packattn_block.h``: what stands around and inside the packed attention in a DiT block.

As in the package's other bindings, the functions named ``pa_*`` mirror the C ABI and only marshal arguments;
the others allocate outputs and scratch memory, call them and raise on a host-side error status.  Outputs and
scratch come from torch's allocator under ``stream`` (default: the current stream of the tensors' device), so
they may be freed or captured into a graph like any other tensor of that stream.  None of them is known to autograd: a
forward call does not record its backward, which is the ``_bwd`` beside it.
"""
import contextlib
import ctypes
import math

NORM_KINDS = {"none": 0, "layer": 1, "rms": 2}


class BlockNormDesc(ctypes.Structure):
    """``pa_block_norm_desc``."""
    _fields_ = [("total_tokens", ctypes.c_int32), ("batch", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("residual_fp32", ctypes.c_int32), ("param_fp32", ctypes.c_int32), ("post", ctypes.c_int32),
                ("pre", ctypes.c_int32), ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("cu_seqlens", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("shift", ctypes.c_void_p), ("gate_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("shift_stride", ctypes.c_int64), ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p)]


class RopeAxesDesc(ctypes.Structure):
    """``pa_rope_axes_desc``."""
    _fields_ = [("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * 4), ("theta", ctypes.c_double * 4),
                ("interleaved", ctypes.c_int32)]


def declare(lib):
    """Sets the argument types of the header's functions on a loaded library."""
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    norm, rope = ctypes.POINTER(BlockNormDesc), ctypes.POINTER(RopeAxesDesc)
    for name, res, args in (
            ("pa_block_norm_fwd", ctypes.c_int, [norm, vp, vp, vp, vp, vp]),
            ("pa_block_norm_workspace_bytes", i64, [i32, i32, i32]),
            ("pa_block_norm_bwd", ctypes.c_int, [norm] + [vp] * 12 + [i64, vp]),
            ("pa_rope_axes", ctypes.c_int, [vp, vp, vp, i32, i32, i32, rope, i32, vp, vp, vp]),
            ("pa_rope_axes_workspace_bytes", i64, [i32, i32]),
            ("pa_qkv_rope_axes_fwd", ctypes.c_int, [vp, vp, vp, i32, i32, i32, i32, rope, vp, vp, vp, vp, i64, vp]),
            ("pa_block_rows", i64, [i32, i32]),
            ("pa_block_select_workspace_bytes", i64, [i32, i32, i32, i32]),
            ("pa_block_select", ctypes.c_int, [vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_double, i32, i32, vp, vp, vp,
                                               i64, vp]),
            ("pa_block_sparse_workspace_bytes", i64, [i32] * 7),
            ("pa_block_sparse_attn_fwd", ctypes.c_int, [vp] * 4 + [i32] * 5 + [vp, vp, i32, f32, vp, vp, vp, i64, vp]),
            ("pa_block_sparse_attn_bwd", ctypes.c_int, [vp] * 7 + [i32] * 5 + [vp, vp, i32, f32, vp, vp, vp, vp, i64,
                                                                               vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


_lib = None


def _library():
    global _lib
    if _lib is None:
        import dit_resolution_packed_b200 as pa
        _lib = pa.load_library()
    return _lib


def _raise_on(rc, where):
    if rc != 0:
        import dit_resolution_packed_b200 as pa
        raise pa.PackAttnError(rc, where)


def _handle(stream, like):
    """cudaStream_t of ``stream``, or of the current stream of the device that ``like`` lives on."""
    if stream is not None:
        return stream.cuda_stream
    if not like.is_cuda:
        return None  # the call refuses host memory
    global _current
    if _current is None:
        import torch
        _current = torch._C._cuda_getCurrentRawStream  # what current_stream() wraps, at a tenth of its time
    return _current(like.get_device())


_current = None
_HERE = contextlib.nullcontext()


def _under(stream):
    if stream is None:
        return _HERE
    import torch
    return torch.cuda.stream(stream)


def _p(t):
    return None if t is None else t.data_ptr()


def _check(dtype, shape, **tensors):
    """Each given tensor is contiguous, of this type and (unless None) of this shape."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _scratch(workspace):
    """Address and bytes of a workspace (none, or a contiguous tensor: an expanded one has fewer bytes than elements)."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- norms, gate and residual

def _norm_desc(like, cu_seqlens, gate, post, w_post, residual_scale, pre, w_pre, scale, shift, eps):
    import torch
    if like.dim() != 2:
        raise ValueError("the residual stream must be [T, C]")
    T, C = like.shape
    f32, bf16 = torch.float32, torch.bfloat16
    if like.dtype is not bf16 and like.dtype is not f32:
        raise TypeError(f"the residual stream must be bfloat16 or float32, got {like.dtype}")
    if post not in NORM_KINDS or pre not in NORM_KINDS:
        raise ValueError(f"post and pre must be one of {sorted(NORM_KINDS)}")
    B = 1  # without cu_seqlens: one segment over all tokens, which nothing reads
    if cu_seqlens is not None:
        _check(torch.int32, None, cu_seqlens=cu_seqlens)
        B = cu_seqlens.numel() - 1
    kind, at, strides = None, [], []
    for name, t in (("gate", gate), ("scale", scale), ("shift", shift), ("w_post", w_post), ("w_pre", w_pre)):
        row = name[0] != "w"  # of an image, or one weight for all
        if t is None:
            at.append(None)
            if row:
                strides.append(0)
            continue
        kind = kind or t.dtype
        if t.dtype is not kind or (kind is not bf16 and kind is not f32):
            raise TypeError("gate, scale, shift and the weights must be all bfloat16 or all float32")
        if row:
            if cu_seqlens is None:
                raise ValueError(f"{name} needs cu_seqlens")
            if t.shape != (B, C) or t.stride(1) != 1:
                raise ValueError(f"{name} must be [B, C] with contiguous rows")
            strides.append(t.stride(0) if B > 1 else 0)
        elif t.shape != (C,) or t.stride(0) != 1:
            raise ValueError(f"{name} must be [C], contiguous")
        at.append(t.data_ptr())
    return BlockNormDesc(T, B, C, like.dtype is f32, kind is f32, NORM_KINDS[post], NORM_KINDS[pre], residual_scale, eps,
                         _p(cu_seqlens), at[0], at[1], at[2], strides[0], strides[1], strides[2], at[3], at[4])


def pa_block_norm_workspace_bytes(batch, total_tokens, hidden):
    """C ``pa_block_norm_workspace_bytes``."""
    return int(_library().pa_block_norm_workspace_bytes(int(batch), int(total_tokens), int(hidden)))


def pa_block_norm_fwd(x, cu_seqlens, y, r, z, *, gate=None, post="none", w_post=None, residual_scale=1.0, pre="none",
                      w_pre=None, scale=None, shift=None, eps=1e-6, stream=None):
    """C ``pa_block_norm_fwd``: x, r [T, C] (bf16 or fp32), y, z bf16 [T, C], gate, scale, shift [B, C] (rows may be
    strided), weights [C]; y, r and z may be None as the header says.  Returns the status code."""
    import torch
    desc = _norm_desc(x, cu_seqlens, gate, post, w_post, residual_scale, pre, w_pre, scale, shift, eps)
    _check(x.dtype, x.shape, x=x, r=r)
    _check(torch.bfloat16, x.shape, y=y, z=z)
    return _library().pa_block_norm_fwd(ctypes.byref(desc), _p(x), _p(y), _p(r), _p(z), _handle(stream, x))


def block_norm_fwd(x, cu_seqlens=None, *, y=None, gate=None, post="none", w_post=None, residual_scale=1.0,
                   pre="layer", w_pre=None, scale=None, shift=None, eps=1e-6, stream=None):
    """The join between two blocks: r = residual_scale x + gate[s] N_post(y) w_post, and the next block's input
    z = N_pre(r) w_pre (1 + scale[s]) + shift[s], s being the image of a token.

    x [T, C] bf16 or fp32; y bf16 [T, C] (None: no join, r is x); gate, scale, shift [B, C] and weights [C], each
    optional; post and pre "none", "layer" or "rms".  Returns (r of x's type, z bf16, or None with pre "none")."""
    import torch
    with _under(stream):
        r = torch.empty_like(x) if y is not None else None
        z = torch.empty_like(x, dtype=torch.bfloat16) if pre != "none" else None
    rc = pa_block_norm_fwd(x, cu_seqlens, y, r, z, gate=gate, post=post, w_post=w_post, residual_scale=residual_scale,
                           pre=pre, w_pre=w_pre, scale=scale, shift=shift, eps=eps, stream=stream)
    _raise_on(rc, "pa_block_norm_fwd")
    return (x if y is None else r), z


def pa_block_norm_bwd(r, cu_seqlens, y, dr, dz, dx, dy, dgate, dscale, dshift, dw_post, dw_pre, workspace, *,
                      gate=None, post="none", w_post=None, residual_scale=1.0, pre="none", w_pre=None, scale=None,
                      shift=None, eps=1e-6, stream=None):
    """C ``pa_block_norm_bwd``: r, dr, dx [T, C] of the residual's type, y, dz, dy bf16 [T, C], dgate, dscale, dshift
    fp32 [B, C], dw_post, dw_pre fp32 [C], workspace a byte tensor; None as the header says."""
    import torch
    desc = _norm_desc(r, cu_seqlens, gate, post, w_post, residual_scale, pre, w_pre, scale, shift, eps)
    _check(r.dtype, r.shape, r=r, dr=dr, dx=dx)
    _check(torch.bfloat16, r.shape, y=y, dz=dz, dy=dy)
    _check(torch.float32, (desc.batch, desc.hidden), dgate=dgate, dscale=dscale, dshift=dshift)
    _check(torch.float32, (desc.hidden,), dw_post=dw_post, dw_pre=dw_pre)
    return _library().pa_block_norm_bwd(
        ctypes.byref(desc), _p(r), _p(y), _p(dr), _p(dz), _p(dx), _p(dy), _p(dgate), _p(dscale), _p(dshift),
        _p(dw_post), _p(dw_pre), *_scratch(workspace), _handle(stream, r))


def block_norm_bwd(r, cu_seqlens=None, dr=None, dz=None, *, y=None, gate=None, post="none", w_post=None,
                   residual_scale=1.0, pre="layer", w_pre=None, scale=None, shift=None, eps=1e-6, stream=None):
    """Gradients of ``block_norm_fwd`` from its r (x where there was no join), dr = dL/dr (or None) and dz = dL/dz,
    with the forward's other arguments.  Returns a dict with dx and, each None where the forward had no such input,
    dy, dgate, dscale, dshift (fp32 [B, C]), dw_post, dw_pre (fp32 [C])."""
    import torch
    C = r.shape[1]
    with _under(stream):
        out = dict(dx=torch.empty_like(r), dy=torch.empty_like(y) if y is not None else None)
        for name, t in (("dgate", gate), ("dscale", scale), ("dshift", shift), ("dw_post", w_post), ("dw_pre", w_pre)):
            out[name] = r.new_empty(t.shape, dtype=torch.float32) if t is not None else None
        ws = None
        if any(t is not None for t in (gate, scale, shift, w_post, w_pre)):
            B = cu_seqlens.numel() - 1 if cu_seqlens is not None else 1
            ws = r.new_empty(max(pa_block_norm_workspace_bytes(B, r.shape[0], C), 0), dtype=torch.uint8)
    rc = pa_block_norm_bwd(r, cu_seqlens, y, dr, dz, out["dx"], out["dy"], out["dgate"], out["dscale"], out["dshift"],
                           out["dw_post"], out["dw_pre"], ws, gate=gate, post=post, w_post=w_post,
                           residual_scale=residual_scale, pre=pre, w_pre=w_pre, scale=scale, shift=shift, eps=eps,
                           stream=stream)
    _raise_on(rc, "pa_block_norm_bwd")
    return out


# ---------------------------------------------------------------- rotary positions with several axes

def _rope_desc(pos, total, dims, theta, interleaved):
    import torch
    dims = [int(n) for n in dims]
    bases = [float(theta)] * len(dims) if isinstance(theta, (int, float)) else [float(b) for b in theta]
    if not 1 <= len(dims) <= 4 or len(bases) != len(dims):
        raise ValueError("dims and theta: 1 to 4 axes, one base or one per axis")
    _check(torch.float32, (total, len(dims)), pos=pos)
    desc = RopeAxesDesc(axes=len(dims), interleaved=int(bool(interleaved)))
    for a, (n, b) in enumerate(zip(dims, bases)):
        desc.dims[a], desc.theta[a] = n, b
    return desc


def pa_rope_axes(q, k, pos, dims, theta, interleaved, inverse, q_out, k_out, stream=None):
    """C ``pa_rope_axes``: q, k (or None), q_out, k_out bf16 [T, H, d], pos fp32 [T, axes].  Returns the status."""
    import torch
    if q.dim() != 3:
        raise ValueError("q must be [T, H, d]")
    _check(torch.bfloat16, q.shape, q=q, k=k, q_out=q_out, k_out=k_out)
    T, H, d = q.shape
    desc = _rope_desc(pos, T, dims, theta, interleaved)
    return _library().pa_rope_axes(_p(q), _p(k), _p(pos), T, H, d, ctypes.byref(desc), int(bool(inverse)), _p(q_out),
                                   _p(k_out), _handle(stream, q))


def _rope_axes(q, k, pos, dims, theta, interleaved, inverse, stream):
    import torch
    with _under(stream):
        q_out = torch.empty_like(q)
        k_out = torch.empty_like(k) if k is not None else None
    _raise_on(pa_rope_axes(q, k, pos, dims, theta, interleaved, inverse, q_out, k_out, stream), "pa_rope_axes")
    return q_out, k_out


def rope_axes_fwd(q, k, pos, dims, theta=10000.0, interleaved=False, stream=None):
    """q and k [T, H, d] turned by positions with several axes: pos fp32 [T, axes]; dims, the channels of each axis
    (their sum at most d, the channels behind them stay); theta one base or one per axis.  k may be None."""
    return _rope_axes(q, k, pos, dims, theta, interleaved, False, stream)


def rope_axes_bwd(dq, dk, pos, dims, theta=10000.0, interleaved=False, stream=None):
    """Gradients of ``rope_axes_fwd``'s inputs from those of its outputs: the inverse rotation."""
    return _rope_axes(dq, dk, pos, dims, theta, interleaved, True, stream)


def pa_rope_axes_workspace_bytes(total_tokens, head_dim):
    """C ``pa_rope_axes_workspace_bytes``."""
    return int(_library().pa_rope_axes_workspace_bytes(int(total_tokens), int(head_dim)))


def pa_qkv_rope_axes_fwd(x, w_qkv, pos, dims, theta, interleaved, q, k, v, workspace, stream=None):
    """C ``pa_qkv_rope_axes_fwd``: x [T, C], w_qkv [3*H*d, C], q, k, v [T, H, d] (bf16), workspace a byte tensor."""
    import torch
    T, C = x.shape
    _, H, d = q.shape
    _check(torch.bfloat16, (T, C), x=x)
    _check(torch.bfloat16, (3 * H * d, C), w_qkv=w_qkv)
    _check(torch.bfloat16, (T, H, d), q=q, k=k, v=v)
    desc = _rope_desc(pos, T, dims, theta, interleaved)
    return _library().pa_qkv_rope_axes_fwd(_p(x), _p(w_qkv), _p(pos), T, C, H, d, ctypes.byref(desc), _p(q), _p(k),
                                           _p(v), *_scratch(workspace), _handle(stream, x))


def qkv_rope_axes_fwd(x, w_qkv, pos, heads, head_dim, dims, theta=10000.0, interleaved=False, stream=None):
    """Fused QKV projection with ``rope_axes_fwd``'s rotation in its epilogue; returns q, k, v bf16 [T, H, d]."""
    import torch
    T = x.shape[0]
    with _under(stream):
        q, k, v = (x.new_empty((T, heads, head_dim)) for _ in range(3))
        ws = x.new_empty(max(pa_rope_axes_workspace_bytes(T, head_dim), 0), dtype=torch.uint8)
    _raise_on(pa_qkv_rope_axes_fwd(x, w_qkv, pos, dims, theta, interleaved, q, k, v, ws, stream),
              "pa_qkv_rope_axes_fwd")
    return q, k, v


# ---------------------------------------------------------------- attention over selected blocks

BLOCK_TOKENS = 128


def pa_block_rows(batch, total_tokens):
    """C ``pa_block_rows``: rows of the block tables of a pack."""
    return int(_library().pa_block_rows(int(batch), int(total_tokens)))


def _pack(cu_seqlens, **tensors):
    """Checks [T, H, d] bf16 tensors of one pack; returns T, H, d, B."""
    import torch
    _check(torch.int32, None, cu_seqlens=cu_seqlens)
    first = next(iter(tensors.values()))
    if first.dim() != 3:
        raise ValueError("q, k and v must be [T, H, d]")
    _check(torch.bfloat16, first.shape, **tensors)
    return tuple(first.shape) + (cu_seqlens.numel() - 1,)


def _lists(idx, cnt, heads, rows):
    import torch
    if idx.dim() != 3:
        raise ValueError("idx must be [H, rows, width]")
    _check(torch.int32, (heads, rows, idx.shape[2]), idx=idx)
    _check(torch.int32, (heads, rows), cnt=cnt)
    return idx.shape[2]


def pa_block_select_workspace_bytes(batch, total_tokens, heads, head_dim):
    """C ``pa_block_select_workspace_bytes``."""
    return int(_library().pa_block_select_workspace_bytes(int(batch), int(total_tokens), int(heads), int(head_dim)))


def pa_block_select(q, k, cu_seqlens, max_seqlen, density, min_blocks, idx, cnt, workspace, stream=None):
    """C ``pa_block_select``: q, k bf16 [T, H, d]; idx int32 [H, rows, width], cnt int32 [H, rows] (written);
    workspace a byte tensor.  Returns the status code."""
    T, H, d, B = _pack(cu_seqlens, q=q, k=k)
    width = _lists(idx, cnt, H, T // BLOCK_TOKENS + B)
    return _library().pa_block_select(_p(q), _p(k), _p(cu_seqlens), B, T, H, d, int(max_seqlen), float(density),
                                      int(min_blocks), width, _p(idx), _p(cnt), *_scratch(workspace), _handle(stream, q))


def block_select(q, k, cu_seqlens, max_seqlen, density, min_blocks=1, stream=None):
    """The key blocks that each block of 128 queries of an image attends to: of the image's nb blocks the
    min(nb, max(min_blocks, ceil(density nb))) whose mean key has the largest product with the mean query.

    Returns idx int32 [H, rows, width] (increasing, -1 behind the list) and cnt int32 [H, rows]; block b of image s
    is row cu_seqlens[s] // 128 + s + b."""
    import torch
    T, H, d = q.shape
    B = cu_seqlens.numel() - 1
    nb = max(1, -(-int(max_seqlen) // BLOCK_TOKENS))
    share = math.ceil(density * nb) if 0.0 <= density <= 1.0 else 0  # (else the call refuses it)
    width = min(nb, max(int(min_blocks), share))
    with _under(stream):
        rows = T // BLOCK_TOKENS + B
        idx = q.new_empty((H, rows, max(width, 1)), dtype=torch.int32)
        cnt = q.new_empty((H, rows), dtype=torch.int32)
        ws = q.new_empty(max(pa_block_select_workspace_bytes(B, T, H, d), 0), dtype=torch.uint8)
    _raise_on(pa_block_select(q, k, cu_seqlens, max_seqlen, density, min_blocks, idx, cnt, ws, stream),
              "pa_block_select")
    return idx, cnt


def pa_block_sparse_workspace_bytes(batch, total_tokens, heads, head_dim, max_seqlen, width, backward):
    """C ``pa_block_sparse_workspace_bytes``."""
    return int(_library().pa_block_sparse_workspace_bytes(int(batch), int(total_tokens), int(heads), int(head_dim),
                                                          int(max_seqlen), int(width), int(bool(backward))))


def pa_block_sparse_attn_fwd(q, k, v, cu_seqlens, max_seqlen, idx, cnt, scale, out, lse, workspace, stream=None):
    """C ``pa_block_sparse_attn_fwd``: q, k, v, out bf16 [T, H, d], lse fp32 [T, H], idx int32 [H, rows, width], cnt
    int32 [H, rows], workspace a byte tensor.  Returns the status code."""
    import torch
    T, H, d, B = _pack(cu_seqlens, q=q, k=k, v=v, out=out)
    _check(torch.float32, (T, H), lse=lse)
    width = _lists(idx, cnt, H, T // BLOCK_TOKENS + B)
    return _library().pa_block_sparse_attn_fwd(_p(q), _p(k), _p(v), _p(cu_seqlens), B, T, H, d, int(max_seqlen),
                                               _p(idx), _p(cnt), width, float(scale), _p(out), _p(lse),
                                               *_scratch(workspace), _handle(stream, q))


def _sparse_workspace(q, cu_seqlens, max_seqlen, idx, backward):
    import torch
    T, H, d = q.shape
    n = pa_block_sparse_workspace_bytes(cu_seqlens.numel() - 1, T, H, d, max(int(max_seqlen), 0), idx.shape[2], backward)
    return q.new_empty(max(n, 0), dtype=torch.uint8)


def block_sparse_attn_fwd(q, k, v, cu_seqlens, max_seqlen, idx, cnt, scale=None, stream=None):
    """``varlen_attn_fwd`` over the key blocks that idx and cnt list (from ``block_select``, or a pattern of the
    caller's).  A query block with an empty list gets out = 0, lse = -inf.  Returns out bf16 [T, H, d], lse [T, H]."""
    import torch
    if scale is None:
        scale = q.shape[-1] ** -0.5
    with _under(stream):
        out = torch.empty_like(q)
        lse = q.new_empty(q.shape[:2], dtype=torch.float32)
        ws = _sparse_workspace(q, cu_seqlens, max_seqlen, idx, False)
    _raise_on(pa_block_sparse_attn_fwd(q, k, v, cu_seqlens, max_seqlen, idx, cnt, scale, out, lse, ws, stream),
              "pa_block_sparse_attn_fwd")
    return out, lse


def pa_block_sparse_attn_bwd(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, idx, cnt, scale, dq, dk, dv, workspace,
                             stream=None):
    """C ``pa_block_sparse_attn_bwd``: tensors as for ``pa_varlen_attn_bwd``, lists and workspace as for
    ``pa_block_sparse_attn_fwd`` (backward = 1).  Returns the status code."""
    import torch
    T, H, d, B = _pack(cu_seqlens, q=q, k=k, v=v, out=out, dout=dout, dq=dq, dk=dk, dv=dv)
    _check(torch.float32, (T, H), lse=lse)
    width = _lists(idx, cnt, H, T // BLOCK_TOKENS + B)
    return _library().pa_block_sparse_attn_bwd(_p(q), _p(k), _p(v), _p(out), _p(lse), _p(dout), _p(cu_seqlens), B, T, H,
                                               d, int(max_seqlen), _p(idx), _p(cnt), width, float(scale), _p(dq),
                                               _p(dk), _p(dv), *_scratch(workspace), _handle(stream, q))


def block_sparse_attn_bwd(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, idx, cnt, scale=None, stream=None):
    """Gradients of ``block_sparse_attn_fwd`` (the lists are constants); returns dq, dk, dv, bf16 [T, H, d]."""
    import torch
    if scale is None:
        scale = q.shape[-1] ** -0.5
    with _under(stream):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = _sparse_workspace(q, cu_seqlens, max_seqlen, idx, True)
    _raise_on(pa_block_sparse_attn_bwd(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, idx, cnt, scale, dq, dk, dv, ws,
                                       stream), "pa_block_sparse_attn_bwd")
    return dq, dk, dv
