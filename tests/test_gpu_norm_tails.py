"""The norm and its gradients where a row is one large value among tiny ones, at the places where threads' pieces meet: a
lost or doubled element changes the root by a constant factor, which no tolerance of a long sum hides. Among them rows of
every odd kind that takes 16 waves, the sum in the residual's place."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors, check, round_to, workspace
from oracle import layers as L
from rows_util import q8_window, row_bytes, unpack
from test_gpu_norm_range import TINY, root_off, terms

pytestmark = pytest.mark.gpu

# a wave to a row with 1, 2 and 4 pieces a lane; 4 and 16 waves; rows past the registers; shorter than a piece
COLS = {"bf16": [3, 9, 77, 511, 513, 1001, 1031, 2047, 2049, 4095, 4101, 8191, 8193, 9001, 12345, 16383, 16385, 24577, 32767, 32771, 70001],
        "f32": [3, 5, 77, 255, 257, 511, 515, 1023, 1025, 2047, 2049, 4095, 4099, 8191, 8195, 9999, 16383, 16387, 40001]}


def _places(cols, piece):
    """Columns of the large value: the ends of the row, of its last whole piece and of the one that starts early, the ends of
    a wave's and a workgroup's shares."""
    last = cols // piece * piece
    at = {0, cols - 1, cols // 2, last, last - 1, cols - piece, cols - piece - 1, cols - piece + 1, 64 * piece - 1, 64 * piece,
          256 * piece - 1, 256 * piece, 1024 * piece - 1, 1024 * piece, 2048 * piece}
    return sorted(c for c in at if 0 <= c < cols)


@pytest.mark.parametrize("dtype,cols", [(d, c) for d in COLS for c in COLS[d]])
def test_one_large_value(dtype, cols):
    say(f"norm: one large value, cols={cols} {dtype}")
    rng = np.random.default_rng(cols)
    at = _places(cols, 4 if dtype == "f32" else 8)
    rows, eps = len(at), float(np.float32(2.0 ** -40))
    spike = np.zeros((1, rows, cols), bool)
    spike[0, range(rows), at] = True
    tiny = lambda: rng.normal(size=(1, rows, cols)) * 2.0 ** -24  # noqa: E731
    x, res = (round_to(np.where(spike, rng.uniform(1, 2, size=spike.shape), tiny()), dtype) for _ in range(2))
    dout = round_to(np.where(spike, rng.uniform(1, 2, size=spike.shape), rng.normal(size=spike.shape) * 2.0 ** -12), dtype)
    dsum = round_to(np.where(spike, 0.0, tiny()), dtype)
    g = round_to(rng.uniform(0.5, 1.5, size=(1, cols)), dtype)
    h = round_to((x.astype(np.float32) + res.astype(np.float32)), dtype)
    shape, half, rel = vr.vrNormShape(DT[dtype], rows, cols, eps), HALF[dtype], root_off(cols, dtype)
    with Job(1) as job:
        tn = Tensors(job, dtype, off=1)
        place, place_read = tn.put(res)
        out, read = tn.put(shape=(rows, cols), fill=5.0)
        q8, q8_read = q8_window(job, (rows, row_bytes(cols)))
        gs = tn.put(g)[0]
        vr.vr_norm(job.comm, shape, tn.put(x)[0], gain=gs, residual=place, sum=place, out=out, q8=q8)
        assert np.array_equal(place_read(), h)
        want = L.norm(h[0], g[0], eps)
        check(read()[0], want, np.abs(want) * (rel + 4 * STEP + half) + TINY, "out")
        values, scales = unpack(q8_read()[0], cols)
        top = np.abs(want).max(-1)
        assert np.all(np.abs(scales - top / 127) <= top / 127 * (rel + 8 * STEP))
        assert np.all(np.abs(values[range(rows), at]) == 127) and not values[~spike[0]].any()

        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        dh, dh_read = tn.put(dsum)  # in dsum's place
        dg, dg_read = tn.put(shape=(cols,), fill=5.0)
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], place, gain=gs, dsum=dh, dh=dh, dgain=dg, workspace=workspace(need),
                            workspace_bytes=need)
        wh, wg = L.norm_backward(dout[0], h[0], g[0], eps, dsum[0])
        root = np.sqrt((h[0] ** 2).mean(-1, keepdims=True) + eps)
        n, w = np.abs(h[0] / root), np.abs(dout[0] * g[0])
        part = (w * (rel + 8 * STEP) + n * (w * n).mean(-1, keepdims=True) * (terms(cols, dtype) * STEP + 2 * rel + 8 * STEP)) / root
        check(dh_read()[0], wh, part + np.abs(wh) * (half + 2 * STEP) + TINY, "dh")
        tol = (np.abs(dout[0]) * n).sum(0) * ((rows + 8) * STEP + rel + 4 * STEP) + np.abs(wg) * half + TINY
        check(dg_read()[0], wg, tol, "dgain")
        job.assert_no_async_error()


@pytest.mark.parametrize("dtype,cols", [("bf16", 1043), ("bf16", 2045), ("f32", 521), ("f32", 1022)])
def test_one_large_value_in_each_of_many_rows(dtype, cols):
    # 16384 rows and more: a wave to a row of 129 to 256 pieces
    import torch
    rows = 16400
    say(f"norm gradients: one large value in each of {rows} rows of {cols} {dtype}")
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    eps, rel, half = float(np.float32(2.0 ** -40)), root_off(cols, dtype), HALF[dtype]
    shape = vr.vrNormShape(DT[dtype], rows, cols, eps)
    gen = torch.Generator(device="cuda").manual_seed(cols)
    places = torch.tensor(_places(cols, 4 if dtype == "f32" else 8), device="cuda")
    spike = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
    spike[torch.arange(rows, device="cuda"), places[torch.arange(rows, device="cuda") % len(places)]] = True
    with Job(1) as job:
        def window(t):
            w, (v,) = job.window(t.numel() * tt.itemsize, fill=0)
            v.view(tt).copy_(t.reshape(-1))
            return vr.vrSlice(w, 0), v.view(tt).view(t.shape)
        large = lambda s: torch.where(spike, 1 + torch.rand(rows, cols, generator=gen, device="cuda"),  # noqa: E731
                                      torch.randn(rows, cols, generator=gen, device="cuda") * s)
        (hs, h), (ds, dout) = window(large(2.0 ** -24)), window(large(2.0 ** -12))
        (dhs, dh), (dgs, dg) = window(torch.zeros(rows, cols, device="cuda")), window(torch.zeros(cols, device="cuda"))
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        vr.vr_norm_backward(job.comm, shape, ds, hs, dh=dhs, dgain=dgs, workspace=workspace(need), workspace_bytes=need)
        torch.cuda.synchronize()
        v, d = h.double(), dout.double()
        root = (v.square().mean(-1, keepdim=True) + eps).sqrt()
        n = v / root
        wh = (d - n * (d * n).mean(-1, keepdim=True)) / root
        part = (d.abs() * (rel + 8 * STEP) + n.abs() * (d * n).abs().mean(-1, keepdim=True)
                * (terms(cols, dtype) * STEP + 2 * rel + 8 * STEP)) / root
        assert bool(((dh.double() - wh).abs() <= part + wh.abs() * (half + 2 * STEP) + TINY).all())
        wg, mag = (d * n).sum(0), (d * n).abs().sum(0)
        # a wave's rows one after the other, four waves, 1024 workgroups by 32 and 32: 17 + 4 + 32 + 32 additions at most
        assert bool(((dg.double() - wg).abs() <= mag * (90 * STEP + rel) + wg.abs() * half + TINY).all())
        job.assert_no_async_error()
