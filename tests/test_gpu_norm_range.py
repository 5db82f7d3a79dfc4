"""The root-mean-square norm and its gradients near the ends of binary32's range, against the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors, check, round_to, workspace
from oracle import layers as L

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126


def terms(cols, dtype):
    """Additions on the longest way into a row's sum: a thread's own elements (32 at most where registers hold the row, else
    every 1024th piece), 6 steps in a wave and 16 waves."""
    piece = 4 if dtype == "f32" else 8
    return max(32, -(-cols // (1024 * piece)) * piece) + 22


def root_off(cols, dtype):
    """Relative error of 1 / root: the squares' sum, of positive terms, halved; the division, eps, the root, its inverse."""
    return terms(cols, dtype) * STEP / 2 + 4 * STEP


@pytest.mark.parametrize("cols", [5, 300, 1000, 3000, 9000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_root_whose_square_passes_binary32(cols, dtype):
    # the squares' sum is finite, and so is eps; the two together are not
    say(f"norm: eps near the largest number, cols={cols} {dtype}")
    rng = np.random.default_rng(cols)
    scale = 2.0 ** np.array([0.0, 40.0, 52.5, 55.0, 62.0])[None, :, None]
    h = round_to(np.clip(rng.normal(size=(1, 5, cols)), -3, 3) * scale, dtype)
    g, dout = round_to(rng.normal(size=(1, cols)), dtype), round_to(rng.normal(size=(1, 5, cols)), dtype)
    eps = float(np.finfo(np.float32).max)
    shape = vr.vrNormShape(DT[dtype], 5, cols, eps)
    rel, half = root_off(cols, dtype), HALF[dtype]
    with Job(1) as job:
        tn = Tensors(job, dtype)
        out, read = tn.put(shape=(5, cols))
        hs, gs = tn.put(h)[0], tn.put(g)[0]
        vr.vr_norm(job.comm, shape, hs, gain=gs, out=out)
        want = L.norm(h[0], g[0], eps)
        check(read()[0], want, np.abs(want) * (rel + 4 * STEP + half) + TINY, "out")
        dh, dh_read = tn.put(shape=(5, cols))
        dg, dg_read = tn.put(shape=(cols,))
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], hs, gain=gs, dh=dh, dgain=dg, workspace=workspace(need),
                            workspace_bytes=need)
        wh, wg = L.norm_backward(dout[0], h[0], g[0], eps)
        root = np.sqrt((h[0] ** 2).mean(-1, keepdims=True) + eps)
        n, w = np.abs(h[0] / root), np.abs(dout[0] * g[0])
        # g and n mean(g n): a sum of cols terms of either sign, and the root's error in each
        part = (w * (rel + 8 * STEP) + n * (w * n).mean(-1, keepdims=True) * (terms(cols, dtype) * STEP + 2 * rel + 8 * STEP)) / root
        check(dh_read()[0], wh, part + np.abs(wh) * (half + 2 * STEP) + TINY, "dh")
        tol = (np.abs(dout[0]) * n).sum(0) * (13 * STEP + rel) + np.abs(wg) * half + TINY
        check(dg_read()[0], wg, tol, "dgain")
        job.assert_no_async_error()


@pytest.mark.parametrize("cols", [5, 300, 3000, 9000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_hold_the_largest_numbers(cols, dtype):
    # as masks have them: the lowest number in a part of a row, in all of it, beside the highest, in the residual alone
    say(f"norm: rows of the largest numbers, cols={cols} {dtype}")
    rng = np.random.default_rng(cols)
    top = float(np.finfo(np.float32).max) if dtype == "f32" else float.fromhex("0x1.fep127")
    x, res = round_to(rng.normal(size=(1, 4, cols)), dtype), np.zeros((1, 4, cols))
    x[0, 0, cols // 2:] = -top
    x[0, 1] = -top
    x[0, 2, ::2], x[0, 2, 1::2] = top, -top
    res[0, 3, 0], x[0, 3, 0] = -top, 0.0
    h = x + res
    g, dout = round_to(rng.normal(size=(1, cols)), dtype), round_to(rng.normal(size=(1, 4, cols)), dtype)
    eps = float(np.float32(1e-5))
    shape = vr.vrNormShape(DT[dtype], 4, cols, eps)
    rel, half = root_off(cols, dtype), HALF[dtype]
    with Job(1) as job:
        tn = Tensors(job, dtype)
        out, read = tn.put(shape=(4, cols))
        total, total_read = tn.put(shape=(4, cols))
        gs = tn.put(g)[0]
        vr.vr_norm(job.comm, shape, tn.put(x)[0], gain=gs, residual=tn.put(res)[0], sum=total, out=out)
        assert np.array_equal(total_read(), h)
        want = L.norm(h[0], g[0], eps)
        check(read()[0], want, np.abs(want) * (rel + 4 * STEP + half) + TINY, "out")
        dh, dh_read = tn.put(shape=(4, cols))
        dg, dg_read = tn.put(shape=(cols,))
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], total, gain=gs, dh=dh, dgain=dg, workspace=workspace(need),
                            workspace_bytes=need)
        wh, wg = L.norm_backward(dout[0], h[0], g[0], eps)
        check(dh_read()[0], wh, TINY, "dh")  # a gradient over 2^127: nothing that is left of it is a normal number
        n = np.abs(L.norm(h[0], None, eps))
        check(dg_read()[0], wg, (np.abs(dout[0]) * n).sum(0) * (12 * STEP + rel) + np.abs(wg) * half + TINY, "dgain")
        job.assert_no_async_error()
