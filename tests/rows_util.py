"""Helpers of the tests of rows in 8 bits: windows of such rows, and what lies in them."""
from __future__ import annotations

import numpy as np

import collective_window_put_amd as vr

GUARD = 0x5A


def row_bytes(cols: int) -> int:
    return (cols + 4 + 127) // 128 * 128


def pack(values, scales) -> np.ndarray:
    """Bytes [..., row bytes] of int8 values [..., cols] and binary32 scales [...]."""
    cols = values.shape[-1]
    got = np.zeros((*values.shape[:-1], row_bytes(cols)), dtype=np.uint8)
    got[..., :cols] = values.view(np.uint8)
    got[..., -4:] = np.ascontiguousarray(scales, dtype=np.float32)[..., None].view(np.uint8)
    return got


def q8_window(job, shape, values=None, off: int = 0):
    """A window of rows of bytes [R, *shape], between guards, `off` bytes in; values: bytes [R, *shape] (else guards).
    Returns (vrSlice, reader of the bytes)."""
    import torch
    n = int(np.prod(shape))
    pad = 256
    h, views = job.window(off + pad + n + pad, fill=None)
    for r, v in enumerate(views):
        v.fill_(GUARD)
        if values is not None:
            v[off + pad:off + pad + n] = torch.from_numpy(np.ascontiguousarray(values[r]).reshape(-1)).cuda()

    def read():
        torch.cuda.synchronize()
        got = []
        for v in views:
            assert bool((v[:off + pad] == GUARD).all()) and bool((v[off + pad + n:] == GUARD).all()), "guard"
            got.append(v[off + pad:off + pad + n].cpu().numpy().reshape(shape))
        return np.stack(got)

    return vr.vrSlice(h, off + pad), read


def unpack(data, cols: int):
    """(int8 values, binary32 scales) of bytes [..., row bytes]; the bytes between are zeros."""
    assert not data[..., cols:-4].any()
    return data[..., :cols].view(np.int8), np.ascontiguousarray(data[..., -4:]).view(np.float32)[..., 0]


def refused(call, code=vr.VR_ERR_INVALID_ARGUMENT):
    import pytest
    with pytest.raises(vr.VrError) as e:
        call()
    assert e.value.code == code
