"""The tensor maps that the kernels write for the segments of a pack are the ones that the encoder would make.

The encoder gives a tensor of less than 131072 bytes another form of map than a larger one.  A short segment's map with the
form of the whole pack's faulted where the tensors lay near the end of mapped memory.  Here every buffer lies in the middle
of a large one, so whatever a map says stays inside mapped memory.
"""
import ctypes
import os
import re

import pytest
import torch

import dit_resolution_packed_b200 as pa
from dit_resolution_packed_b200 import _build

MARGIN = 4 << 20


def _encoded(ptr, rows, channels):
    """128 bytes: the encoder's map of a bf16 [rows, channels] matrix, box 64 x 128, 128-byte swizzle."""
    raw = (ctypes.c_uint8 * 256)()
    at = (ctypes.addressof(raw) + 63) // 64 * 64
    rc = ctypes.CDLL("libcuda.so.1").cuTensorMapEncodeTiled(
        ctypes.c_void_p(at), 9, 2, ctypes.c_void_p(ptr), (ctypes.c_uint64 * 2)(channels, rows),
        (ctypes.c_uint64 * 1)(channels * 2), (ctypes.c_uint32 * 2)(64, 128), (ctypes.c_uint32 * 2)(1, 1), 0, 3, 3, 0)
    assert rc == 0
    return ctypes.string_at(at, 128)


class _Arena:
    def __init__(self, dev):
        self.whole = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
        self.at = MARGIN

    def take(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        t = self.whole[self.at:self.at + n].view(dtype).view(shape)
        self.at += (n + (1 << 17) + 511) // 512 * 512
        assert self.at < self.whole.numel() - MARGIN
        return t


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,d", [
    ([300, 40], 2, 128),               # 150 kB and 20 kB
    ([255, 256, 257, 1], 2, 128),      # one row below the border, and above
    ([1023, 1024, 3, 0, 700], 1, 64),  # the same with rows of 128 bytes
    ([300, 40], 2, 64),                # all of it below
    ([21, 22, 500], 24, 128),          # rows of 6144 bytes
])
def test_segment_maps_are_the_encoders(cuda_device, lens, H, d):
    a = _Arena(cuda_device)
    T, B, longest = sum(lens), len(lens), max(lens)
    starts = [sum(lens[:s]) for s in range(B + 1)]
    q, k, v, dout, out, dq, dk, dv = (a.take((T, H, d), torch.bfloat16) for _ in range(8))
    lse = a.take((T, H), torch.float32)
    for t in (q, k, v, dout):
        t.normal_()
    cu = torch.tensor(starts, dtype=torch.int32, device=cuda_device)
    rows = pa.pa_block_rows(B, T)
    idx = torch.zeros(H, rows, 1, dtype=torch.int32, device=cuda_device)
    cnt = torch.ones(H, rows, dtype=torch.int32, device=cuda_device)
    for backward in (False, True):
        ws = a.take((pa.pa_block_sparse_workspace_bytes(B, T, H, d, longest, 1, backward),), torch.uint8)
        if backward:
            rc = pa.pa_block_sparse_attn_bwd(q, k, v, out, lse, dout, cu, longest, idx, cnt, 0.1, dq, dk, dv, ws)
        else:
            rc = pa.pa_block_sparse_attn_fwd(q, k, v, cu, longest, idx, cnt, 0.1, out, lse, ws)
        assert rc == pa.PA_OK and pa.pa_get_error() == pa.PA_OK
        held = bytes(ws.cpu().numpy())
        for s, n in enumerate(lens):
            for name, t in (("q", q), ("k", k), ("v", v)) + ((("dout", dout),) if backward else ()):
                want = _encoded(t.data_ptr() + starts[s] * H * d * 2, n, H * d) if n else None
                assert want is None or want in held, f"segment {s} of {n} tokens: {name}, backward {backward}"


def test_every_map_is_written_in_one_place():
    """Base and extent are replaced by write_part_map alone, which takes the template of the part's size."""
    found = []
    for name in _build.SOURCES + _build.HEADERS:
        with open(os.path.join(_build.CSRC, name)) as f:
            src = re.sub(r"//[^\n]*", "", f.read())
        found += [name] * src.count("tensormap.replace")
        # whoever encodes a template encodes its small form too
        assert len(re.findall(r"encode_\w+\(&\w+\.tmpl\[", src)) == len(re.findall(r"encode_\w+\(&\w+\.small\[", src)), name
    assert found == ["sm100_ptx.cuh"] * 2
