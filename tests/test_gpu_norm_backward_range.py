"""Gradients of the root-mean-square norm whose sum of g * h passes binary32 while the gradient itself does not, against
the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors, check, round_to, workspace
from oracle import layers as L
from test_gpu_norm_range import TINY, root_off, terms

pytestmark = pytest.mark.gpu

# sizes of a row's h and dout: ordinary ones; products that pass 2^128; the products' sum alone; the sum over the root, of
# small h; squares that pass 2^128 beside dout that do and do not; dout near the largest number
SIZES = [(0, 0), (17, 113), (0, 118), (-12, 112), (64, 3), (100, 120), (20, 124), (64, -60)]


def _back_check(got_h, got_g, dout, h, g, eps, dsum, dtype, what):
    rows, cols = h.shape
    rel, half = root_off(cols, dtype), HALF[dtype]
    wh, wg = L.norm_backward(dout, h, g, eps, dsum)
    root = np.sqrt((h ** 2).mean(-1, keepdims=True) + eps)
    n, w = np.abs(h / root), np.abs(dout * (1.0 if g is None else g))
    # g and n mean(g n): a sum of terms of either sign, and the root's error in each
    part = (w * (rel + 8 * STEP) + n * (w * n).mean(-1, keepdims=True) * (terms(cols, dtype) * STEP + 2 * rel + 8 * STEP)) / root
    check(got_h, wh, part + np.abs(wh) * (half + 2 * STEP) + TINY, what + " dh")
    check(got_g, wg, (np.abs(dout) * n).sum(0) * ((rows + 8) * STEP + rel) + np.abs(wg) * half + TINY, what + " dgain")


@pytest.mark.parametrize("cols", [3, 200, 777, 1500, 4100, 9001, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gain", [True, False])
def test_products_that_pass_binary32(cols, dtype, gain):
    say(f"norm gradients: large g * h, cols={cols} {dtype} gain={gain}")
    rng = np.random.default_rng(cols)
    rows = len(SIZES)
    by = 2.0 ** np.array(SIZES, np.float64)
    clipped = lambda: np.clip(rng.normal(size=(1, rows, cols)), -3, 3)  # noqa: E731
    h, dout = round_to(clipped() * by[None, :, :1], dtype), round_to(clipped() * by[None, :, 1:], dtype)
    g = round_to(rng.uniform(0.5, 1.5, size=(1, cols)), dtype) if gain else None
    dsum = round_to(rng.normal(size=(1, rows, cols)), dtype)
    shape = vr.vrNormShape(DT[dtype], rows, cols, 1e-5)
    eps = float(np.float32(1e-5))
    with Job(1) as job:
        tn = Tensors(job, dtype)
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        dh, dh_read = tn.put(shape=(rows, cols), fill=5.0)
        dg, dg_read = tn.put(shape=(cols,), fill=5.0)
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], tn.put(h)[0], gain=tn.put(g)[0] if gain else None,
                            dsum=tn.put(dsum)[0], dh=dh, dgain=dg, workspace=workspace(need), workspace_bytes=need)
        _back_check(dh_read()[0], dg_read()[0], dout[0], h[0], None if g is None else g[0], eps, dsum[0], dtype, f"cols={cols}")
        job.assert_no_async_error()


def test_such_rows_among_many():
    # a wave to a row: 130 pieces, 16384 rows; the others come out as without them
    import torch
    rows, cols, dtype = 16384, 1040, "bf16"
    say(f"norm gradients: large g * h among {rows} rows")
    shape = vr.vrNormShape(DT[dtype], rows, cols, 1e-5)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    at = sorted(rng.choice(rows, size=len(SIZES), replace=False).tolist())
    with Job(1) as job:
        def window(n, random=True):
            w, (v,) = job.window(n * 2, fill=0)
            t = v.view(torch.bfloat16)
            if random:
                t.copy_(torch.randn(n, generator=gen, device="cuda"))
            return vr.vrSlice(w, 0), t
        (hs, h), (ds, dout), (gs, g), (dhs, dh) = window(rows * cols), window(rows * cols), window(cols), window(rows * cols, False)
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        ws = workspace(need)
        run = lambda: vr.vr_norm_backward(job.comm, shape, ds, hs, gain=gs, dh=dhs, workspace=ws, workspace_bytes=need)  # noqa: E731
        run()
        before = dh.clone().view(rows, cols)
        h, dout = h.view(rows, cols), dout.view(rows, cols)
        for i, (a, b) in zip(at, SIZES):
            h[i] = (h[i].float().clamp(-3, 3) * 2.0 ** a).bfloat16()
            dout[i] = (dout[i].float().clamp(-3, 3) * 2.0 ** b).bfloat16()
        run()
        got = dh.view(rows, cols)
        f = lambda t: t[at].double().cpu().numpy()  # noqa: E731
        hr, dr, gr, eps = f(h), f(dout), g.double().cpu().numpy(), float(np.float32(1e-5))
        wh, _ = L.norm_backward(dr, hr, gr, eps)
        rel = root_off(cols, dtype)
        root = np.sqrt((hr ** 2).mean(-1, keepdims=True) + eps)
        n, w = np.abs(hr / root), np.abs(dr * gr)
        part = (w * (rel + 8 * STEP) + n * (w * n).mean(-1, keepdims=True) * (terms(cols, dtype) * STEP + 2 * rel + 8 * STEP)) / root
        check(f(got), wh, part + np.abs(wh) * (HALF[dtype] + 2 * STEP) + TINY, "dh")
        others = torch.ones(rows, dtype=torch.bool, device="cuda")
        others[at] = False
        assert torch.equal(got[others], before[others])
        job.assert_no_async_error()


@pytest.mark.parametrize("cols", [40, 3000, 9000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [0, 70])
def test_a_dout_that_is_no_number_stays_in_its_row_and_column(cols, dtype, size):
    say(f"norm gradients: an infinite dout, cols={cols} {dtype} h of 2^{size}")
    rng = np.random.default_rng(cols)
    h = round_to(np.clip(rng.normal(size=(1, 3, cols)), -3, 3) * 2.0 ** size, dtype)
    dout = round_to(rng.normal(size=(1, 3, cols)), dtype)
    dout[0, 1, cols // 2] = np.inf
    shape = vr.vrNormShape(DT[dtype], 3, cols, 1e-5)
    eps, rel = float(np.float32(1e-5)), root_off(cols, dtype)
    with Job(1) as job:
        tn = Tensors(job, dtype)
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        dh, dh_read = tn.put(shape=(3, cols), fill=5.0)
        dg, dg_read = tn.put(shape=(cols,), fill=5.0)
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], tn.put(h)[0], dh=dh, dgain=dg, workspace=workspace(need),
                            workspace_bytes=need)
        got, gain = dh_read()[0], dg_read()[0]
        assert not np.isfinite(got[1]).any() and np.isfinite(got[[0, 2]]).all()
        n = h[0] / np.sqrt((h[0] ** 2).mean(-1, keepdims=True) + eps)
        others = np.arange(cols) != cols // 2
        assert not np.isfinite(gain[cols // 2])
        want, mag = (dout[0, :, others] * n[:, others].T).sum(1), (np.abs(dout[0, :, others]) * np.abs(n[:, others].T)).sum(1)
        check(gain[others], want, mag * (11 * STEP + rel) + np.abs(want) * HALF[dtype] + TINY, "dgain")
        job.assert_no_async_error()


@pytest.mark.parametrize("cols", [8, 520, 4100, 20000])
def test_the_largest_g_beside_a_mean_of_the_other_sign(cols):
    # g_0 - n_0 mean passes binary32 by a step, where the gradient, over the root, does not
    say(f"norm gradients: the largest g, cols={cols}")
    h = np.full((1, 1, cols), 2.0)
    h[0, 0, 0] = 0.25
    n = h[0, 0] / np.sqrt((h[0, 0] ** 2).mean())
    dout = np.empty((1, 1, cols))
    dout[0, 0, 0] = float(np.finfo(np.float32).max)
    dout[0, 0, 1:] = (-2.0 ** 114 * cols - dout[0, 0, 0] * n[0]) / n[1:].sum()
    dout = round_to(dout, "f32")
    shape = vr.vrNormShape(DT["f32"], 1, cols, 1e-5)
    with Job(1) as job:
        tn = Tensors(job, "f32")
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        dh, dh_read = tn.put(shape=(1, cols), fill=5.0)
        dg, dg_read = tn.put(shape=(cols,), fill=5.0)
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], tn.put(h)[0], dh=dh, dgain=dg, workspace=workspace(need),
                            workspace_bytes=need)
        _back_check(dh_read()[0], dg_read()[0], dout[0], h[0], None, float(np.float32(1e-5)), None, "f32", f"cols={cols}")
        job.assert_no_async_error()
