"""Helpers of the layer tests: tensors in windows, and the steps of the
element types from which the tolerances are counted."""
from __future__ import annotations

import numpy as np

import collective_window_put_amd as vr
from gpu_util import ALIGN

ACT = {"none": vr.VR_ACT_NONE, "relu": vr.VR_ACT_RELU, "gelu": vr.VR_ACT_GELU, "silu": vr.VR_ACT_SILU}
DT = {"f32": vr.VR_DT_F32, "bf16": vr.VR_DT_BF16}
# half a step of a rounding to the type, relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
# one binary32 addition or matrix-instruction accumulation: at most a whole step (it may truncate)
STEP = 2.0 ** -23
# an activation in binary32: exp, erf, one division and a few products, each within 4 steps of a value that is at
# most max(1, |z|); exp(-z) also carries the argument's rounding, |z| / 2 steps, damped by exp(-|z|) |z| <= 0.4
ACT_EVAL = 2.0 ** -19


def round_to(a, dtype: str) -> np.ndarray:
    """The float64 values of `a` rounded to the type."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64))
    return t.to(torch.float32 if dtype == "f32" else torch.bfloat16).double().numpy()


class Tensors:
    """Windows of a Job with numpy values in and out; `off` shifts every tensor by that many elements."""

    def __init__(self, job, dtype: str, off: int = 0):
        import torch
        self.torch, self.job, self.dtype = torch, job, dtype
        self.tt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.es = 4 if dtype == "f32" else 2
        self.off = off

    def put(self, values=None, shape=None, fill=0.0):
        """A window holding values [R, ...] (or `fill`, of shape per rank); returns (vrSlice, reader)."""
        torch, R = self.torch, self.job.R
        if values is not None:
            shape = values.shape[1:]
        n = int(np.prod(shape))
        pad = 8  # guard elements on both sides stay untouched
        total = self.off + pad + n + pad
        h, views = self.job.window(total * self.es, fill=None)
        for r, v in enumerate(views):
            t = v.view(self.tt)
            t.fill_(7.0)
            t[self.off + pad:self.off + pad + n] = (
                torch.from_numpy(np.ascontiguousarray(values[r], dtype=np.float64)).reshape(-1).to("cuda").to(self.tt)
                if values is not None else fill)

        def read():
            torch.cuda.synchronize()
            got = []
            for v in views:
                t = v.view(self.tt)
                assert bool((t[:self.off + pad] == 7.0).all()) and bool((t[self.off + pad + n:] == 7.0).all()), "guard"
                got.append(t[self.off + pad:self.off + pad + n].double().cpu().numpy().reshape(shape))
            return np.stack(got)

        return vr.vrSlice(h, (self.off + pad) * self.es), read


def workspace(nbytes: int):
    import torch
    return torch.full((max(nbytes, 1) + 256,), 0xFF, dtype=torch.uint8, device="cuda")[:max(nbytes, 1)] if nbytes else None


def check(got, want, tol, what: str):
    """Element by element; NaN nowhere."""
    d = np.abs(got - want)
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], np.broadcast_to(tol, d.shape)[bad][:4],
                           np.argwhere(bad)[:4].tolist())


__all__ = ["ACT", "DT", "HALF", "STEP", "ACT_EVAL", "ALIGN", "round_to", "Tensors", "workspace", "check"]
