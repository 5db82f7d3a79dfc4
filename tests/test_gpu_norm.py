"""The root-mean-square norm and its gradients on the GPU against the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors, check, round_to, workspace
from oracle import layers as L
from rows_util import GUARD, q8_window, refused, row_bytes, unpack

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -130


def _sum(x, residual, dtype):
    """x + residual in binary32, rounded to the type: what the kernel stores, bit for bit."""
    import torch
    if residual is None:
        return x
    t = torch.from_numpy(x).float() + torch.from_numpy(residual).float()
    return (t if dtype == "f32" else t.bfloat16()).double().numpy()


CASES = [  # R, rows, cols, dtype, residual, gain, off
    (1, 1, 1, "f32", False, True, 0),
    (1, 1, 1, "bf16", True, True, 1),
    (2, 3, 7, "bf16", True, False, 3),
    (1, 1, 4096, "bf16", True, True, 0),
    (3, 5, 64, "f32", True, True, 0),
    (2, 9, 77, "f32", True, True, 1),
    (1, 70, 256, "bf16", False, True, 0),
    (1, 33, 260, "f32", True, True, 0),
    (8, 17, 512, "bf16", True, True, 0),
    (1, 6, 520, "bf16", True, True, 1),
    (2, 10, 1001, "bf16", True, True, 0),
    (1, 4, 1024, "f32", False, False, 0),
    (1, 5, 2048, "bf16", True, True, 0),
    (2, 3, 2049, "bf16", False, True, 5),
    (1, 4, 2100, "f32", True, True, 2),
    (1, 3, 4097, "f32", True, True, 0),
    (1, 3, 8192, "bf16", True, True, 0),
    (1, 2, 8200, "bf16", True, True, 1),
    (2, 2, 16384, "f32", True, True, 0),
    (1, 2, 32768, "bf16", True, True, 0),
    (1, 2, 32770, "bf16", True, True, 0),   # past the registers
    (2, 2, 40001, "f32", True, True, 1),
    (1, 2, 70000, "bf16", False, True, 0),
]


@pytest.mark.parametrize("R,rows,cols,dtype,residual,gain,off", CASES)
def test_norm_and_gradients(R, rows, cols, dtype, residual, gain, off):
    say(f"norm R={R} rows={rows} cols={cols} {dtype} residual={residual} gain={gain} off={off}")
    rng = np.random.default_rng(rows + cols)
    f = lambda *s: round_to(rng.normal(size=s), dtype)  # noqa: E731
    size = 10.0 ** rng.uniform(-3, 3, size=(R, rows, 1))  # rows of all sizes
    x, res = round_to(f(R, rows, cols) * size, dtype), round_to(f(R, rows, cols) * size, dtype) if residual else None
    g = f(R, cols) if gain else None
    dout, dsum = f(R, rows, cols), f(R, rows, cols) if residual else None
    eps, half = 2.0 ** -17, HALF[dtype]
    shape = vr.vrNormShape(DT[dtype], rows, cols, eps)
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        put = lambda v: None if v is None else tn.put(v)[0]  # noqa: E731
        xs, rs, gs = put(x), put(res), put(g)
        out, out_read = tn.put(shape=(rows, cols), fill=5.0)
        total, total_read = tn.put(shape=(rows, cols), fill=5.0) if residual else (None, None)
        q8, q8_read = q8_window(job, (rows, row_bytes(cols)), off=4 * off)
        vr.vr_norm(job.comm, shape, xs, gain=gs, residual=rs, sum=total, out=out, q8=q8)
        got, data = out_read(), q8_read()
        h = _sum(x, res, dtype)
        if residual:
            assert np.array_equal(total_read(), h)
        values, scales = unpack(data, cols)
        # the squares' sum: cols + 4 additions at most of positive terms, halved by the root; then the division, the
        # root, and three roundings of the products
        rel = (cols + 4) * STEP / 2 + 8 * STEP
        for r in range(R):
            want = L.norm(h[r], None if g is None else g[r], eps)
            check(got[r], want, np.abs(want) * (rel + half) + TINY, "out")
            top = np.abs(want).max(-1)
            assert np.all(np.abs(scales[r] - top / 127) <= top / 127 * (rel + 4 * STEP) + TINY)
            s = scales[r].astype(np.float64)[:, None]
            # half a step of the scale; its own rounding and the multiplier's, at most 127 times
            check(values[r] * s, want, s * (0.5 + 127 * 4 * STEP) + np.abs(want) * rel + TINY, "q8")

        # one output at a time gives the same; the sum in the residual's place
        out2, out2_read = tn.put(shape=(rows, cols), fill=5.0)
        vr.vr_norm(job.comm, shape, xs, gain=gs, residual=rs, out=out2)
        assert np.array_equal(out2_read(), got)
        q82, q82_read = q8_window(job, (rows, row_bytes(cols)), off=4 * off)
        if residual:
            place, place_read = tn.put(res)
            vr.vr_norm(job.comm, shape, xs, gain=gs, residual=place, sum=place, q8=q82)
            assert np.array_equal(place_read(), h)
        else:
            vr.vr_norm(job.comm, shape, xs, gain=gs, q8=q82)
        assert np.array_equal(q82_read(), data)

        # the gradients
        need = vr.vr_norm_backward_workspace_bytes(R, shape)
        ws = workspace(need)
        dh, dh_read = tn.put(shape=(rows, cols), fill=5.0)
        dg, dg_read = tn.put(shape=(cols,), fill=5.0)
        ds, ss = put(dout), put(dsum)
        hs = put(h)
        vr.vr_norm_backward(job.comm, shape, ds, hs, gain=gs, dsum=ss, dh=dh, dgain=dg, workspace=ws, workspace_bytes=need)
        gh, gg = dh_read(), dg_read()
        for r in range(R):
            gr = None if g is None else g[r]
            wh, wg = L.norm_backward(dout[r], h[r], gr, eps, None if dsum is None else dsum[r])
            root = np.sqrt((h[r] ** 2).mean(-1, keepdims=True) + eps)
            n, w = np.abs(h[r] / root), np.abs(dout[r] * (1.0 if gr is None else gr))
            # g and n mean(g n): a sum of cols terms, and the root's error in each
            part = (w * (rel + 8 * STEP) + n * (w * n).mean(-1, keepdims=True) * ((cols + 4) * STEP + 2 * rel + 8 * STEP)) / root
            check(gh[r], wh, part + np.abs(wh) * (half + 2 * STEP) + TINY, "dh")
            tol = (np.abs(dout[r]) * n).sum(0) * ((rows + 8) * STEP + rel) + np.abs(wg) * half + TINY
            check(gg[r], wg, tol, "dgain")
        # either alone; dh in dsum's place; twice the same
        dg2, dg2_read = tn.put(shape=(cols,), fill=5.0)
        vr.vr_norm_backward(job.comm, shape, ds, hs, gain=gs, dgain=dg2, workspace=ws, workspace_bytes=need)
        assert np.array_equal(dg2_read(), gg)
        place, place_read = tn.put(dsum) if residual else tn.put(shape=(rows, cols))
        vr.vr_norm_backward(job.comm, shape, ds, hs, gain=gs, dsum=place if residual else None, dh=place, workspace=ws,
                            workspace_bytes=need)
        assert np.array_equal(place_read(), gh)
        job.assert_no_async_error()


@pytest.mark.parametrize("R,rows,cols,dtype", [(1, 2500, 96, "bf16"), (3, 1100, 300, "f32"), (1, 3000, 1000, "bf16"),
                                               (8, 300, 2048, "bf16"), (1, 700, 8200, "bf16")])
def test_gain_gradient_over_many_rows(R, rows, cols, dtype):
    say(f"norm gradient: many rows R={R} rows={rows} cols={cols} {dtype}")
    rng = np.random.default_rng(cols)
    h, dout, g = (round_to(rng.normal(size=s), dtype) for s in ((R, rows, cols), (R, rows, cols), (R, cols)))
    shape = vr.vrNormShape(DT[dtype], rows, cols, 1e-5)
    with Job(R) as job:
        tn = Tensors(job, dtype)
        need = vr.vr_norm_backward_workspace_bytes(R, shape)
        dg, read = tn.put(shape=(cols,))
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], tn.put(h)[0], gain=tn.put(g)[0], dgain=dg,
                            workspace=workspace(need), workspace_bytes=need)
        got = read()
        rel = (cols + 4) * STEP / 2 + 16 * STEP
        for r in range(R):
            _, want = L.norm_backward(dout[r], h[r], g[r], 1e-5)
            n = np.abs(L.norm(h[r], None, 1e-5))
            check(got[r], want, (np.abs(dout[r]) * n).sum(0) * ((rows + 8) * STEP + rel) + np.abs(want) * HALF[dtype] + TINY, "dgain")


@pytest.mark.parametrize("cols", [9, 500, 3000, 9000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_huge_and_tiny_values(cols, dtype):
    # squares that pass binary32, and ones below it: the root is the same as of the row times a power of two
    say(f"norm: huge and tiny rows, cols={cols} {dtype}")
    rng = np.random.default_rng(cols)
    base = round_to(np.clip(rng.normal(size=(1, 6, cols)), -3, 3), dtype)
    scale = 2.0 ** np.array([125.0, 90.0, 64.0, 0.0, -60.0, -100.0])[None, :, None]
    h = base * scale
    g, dout = round_to(rng.normal(size=(1, cols)), dtype), round_to(rng.normal(size=(1, 6, cols)), dtype)
    eps = 2.0 ** -126
    shape = vr.vrNormShape(DT[dtype], 6, cols, eps)
    rel = (cols + 4) * STEP / 2 + 8 * STEP
    with Job(1) as job:
        tn = Tensors(job, dtype)
        out, read = tn.put(shape=(6, cols))
        dh, dh_read = tn.put(shape=(6, cols))
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        hs, gs = tn.put(h)[0], tn.put(g)[0]
        vr.vr_norm(job.comm, shape, hs, gain=gs, out=out)
        want = L.norm(h[0], g[0], eps)
        # below 2^-60 the squares leave binary32's normal numbers; there eps holds the root, 2^-63, up
        tol = np.abs(want) * (rel + HALF[dtype]) + 2.0 ** -126
        check(read()[0][:5], want[:5], tol[:5], "out")
        check(read()[0][5], want[5], np.abs(want[5]) * (rel + HALF[dtype] + 2.0 ** -20) + 2.0 ** -126, "tiny")
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], hs, gain=gs, dh=dh, workspace=workspace(need), workspace_bytes=need)
        wh, _ = L.norm_backward(dout[0], h[0], g[0], eps)
        root = np.sqrt((h[0] ** 2).mean(-1, keepdims=True) + eps)
        n, w = np.abs(h[0] / root), np.abs(dout[0] * g[0])
        part = (w * (rel + 8 * STEP) + n * (w * n).mean(-1, keepdims=True) * ((cols + 4) * STEP + 2 * rel + 8 * STEP)) / root
        check(dh_read()[0][:4], wh[:4], (part + np.abs(wh) * (HALF[dtype] + 2 * STEP) + 2.0 ** -126)[:4], "dh")
        job.assert_no_async_error()


@pytest.mark.parametrize("cols", [5, 700, 4100, 33000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_with_values_that_are_no_numbers(cols, dtype):
    say(f"norm: NaN and infinities, cols={cols} {dtype}")
    rng = np.random.default_rng(cols)
    h = round_to(rng.normal(size=(1, 5, cols)), dtype)
    h[0, 1, cols // 2] = np.nan
    h[0, 2, cols - 1] = np.inf
    h[0, 3] = 0.0
    shape = vr.vrNormShape(DT[dtype], 5, cols, 1e-5)
    with Job(1) as job:
        tn = Tensors(job, dtype)
        out, read = tn.put(shape=(5, cols))
        q8, q8_read = q8_window(job, (5, row_bytes(cols)))
        hs = tn.put(h)[0]
        vr.vr_norm(job.comm, shape, hs, out=out, q8=q8)
        assert job.async_error()[1] == vr.VR_ASYNC_BAD_VALUE
        got = read()[0]
        assert np.isnan(got[1]).all() and np.all(got[3] == 0)
        assert np.isnan(got[2, cols - 1]) and np.all(got[2, :cols - 1] == 0)  # h / infinity
        values, scales = unpack(q8_read()[0], cols)
        assert np.isnan(scales[1]) and np.isnan(scales[2]) and scales[3] == 0 and not values[1:4].any()
        assert np.isfinite(scales[[0, 4]]).all() and np.all(np.abs(values[[0, 4]]).max(-1) == 127)
        for i in (0, 4):  # the others are as if alone
            check(got[i], L.norm(h[0, i:i + 1], None, 1e-5)[0], np.abs(got[i]) * (HALF[dtype] * 1.1 + cols * STEP) + TINY, "out")
        vr.vr_norm(job.comm, shape, hs, out=out)
        job.assert_no_async_error()  # without rows in 8 bits nothing is reported


def test_gradient_against_differences():
    say("norm gradient against differences")
    rng = np.random.default_rng(5)
    rows, cols, step = 4, 12, 2.0 ** -8
    x, g, dout = (round_to(rng.normal(size=s), "f32") for s in ((1, rows, cols), (1, cols), (1, rows, cols)))
    shape = vr.vrNormShape(vr.VR_DT_F32, rows, cols, 0.01)
    need = vr.vr_norm_backward_workspace_bytes(1, shape)
    with Job(1) as job:
        tn = Tensors(job, "f32")

        def run(x, g):
            out, read = tn.put(shape=(rows, cols))
            vr.vr_norm(job.comm, shape, tn.put(x)[0], gain=tn.put(g)[0], out=out)
            return float((read() * dout).sum())

        dh, dh_read = tn.put(shape=(rows, cols))
        dg, dg_read = tn.put(shape=(cols,))
        vr.vr_norm_backward(job.comm, shape, tn.put(dout)[0], tn.put(x)[0], gain=tn.put(g)[0], dh=dh, dgain=dg,
                            workspace=workspace(need), workspace_bytes=need)
        for key, grad in (("x", dh_read()), ("g", dg_read())):
            v = rng.normal(size=grad.shape)
            a, b = ((round_to(x + s * step * v, "f32"), g) if key == "x" else (x, round_to(g + s * step * v, "f32")) for s in (1, -1))
            slope = (run(*a) - run(*b)) / (2 * step)
            size = float(np.abs(dout).sum() * np.abs(g).max() * 3.5)
            # the forward's rounding over the step; the third derivative, below 40 |v|^3 / root^3 in these units, times step^2
            assert abs(slope - float((grad * v).sum())) <= size * 64 * STEP / step + 40 * step ** 2 * float((v ** 2).sum()) ** 1.5, key


def test_no_rows_and_refusals():
    import torch
    say("norm: no rows, refusals")
    R, rows, cols = 2, 6, 24
    N = vr.vrNormShape
    with Job(R) as job:
        tn = Tensors(job, "f32")
        t = lambda *s: tn.put(shape=s)[0]  # noqa: E731
        x, res, out, gain = t(rows, cols), t(rows, cols), t(rows, cols), t(cols)
        q8, _ = q8_window(job, (rows, row_bytes(cols)))
        ok = N(vr.VR_DT_F32, rows, cols, 1e-5)
        norm = lambda s, *a, **k: (lambda: vr.vr_norm(job.comm, s, *a, **k))  # noqa: E731
        for bad in (N(2, rows, cols, 1e-5), N(0, -1, cols, 1e-5), N(0, rows, 0, 1e-5), N(0, rows, cols, 0.0),
                    N(0, rows, cols, float("nan")), N(0, rows + 64, cols, 1e-5), N(0, (1 << 24) + 1, cols, 1e-5)):
            refused(norm(bad, x, out=out))
        refused(norm(ok, None, out=out))
        refused(norm(ok, x))                                         # nothing wanted
        refused(norm(ok, x, residual=res, sum=res))
        refused(norm(ok, x, sum=res, out=out))                       # a sum of nothing
        refused(norm(ok, x, out=x))
        refused(norm(ok, x, out=gain, gain=gain))
        refused(norm(ok, x, residual=res, sum=x, out=out))
        refused(norm(ok, x, residual=res, sum=(res.window, res.offset + 4), out=out))
        refused(norm(ok, x, residual=res, sum=out, out=out))
        refused(norm(ok, x, out=out, q8=(out.window, out.offset)))
        refused(norm(ok, x, q8=(q8.window, q8.offset + 2)))
        refused(norm(ok, x, out=(out.window, out.offset + 2)))
        refused(norm(ok, x, q8=(q8.window, q8.offset + 128 * rows)))  # past the window
        sw, _ = job.window(4096, flags=vr.VR_WIN_STRICT_ORDERING)
        vr.vr_va_signal_reset(job.comm, sw, 0, 64)
        refused(norm(ok, x, out=(sw, 0)), vr.VR_ERR_INVALID_USAGE)

        need = vr.vr_norm_backward_workspace_bytes(R, ok)
        ws = workspace(need)
        dh, dg = t(rows, cols), tn.put(shape=(cols,), fill=5.0)
        back = lambda *a, w=ws, n=need, s=ok, **k: (lambda: vr.vr_norm_backward(job.comm, s, *a, workspace=w, workspace_bytes=n, **k))  # noqa: E731
        refused(back(out, x))
        refused(back(None, x, dh=dh))
        refused(back(out, None, dh=dh))
        refused(back(out, x, dh=dh, n=need - 1))
        refused(back(out, x, dh=dh, w=None))
        refused(back(out, x, dh=dh, w=ws[8:]))
        refused(back(out, x, dh=dh, w=torch.zeros(need + 256, dtype=torch.uint8)))  # host memory
        refused(back(out, x, dh=x))
        refused(back(out, x, dh=out))
        refused(back(out, x, gain=gain, dh=dh, dgain=gain))
        refused(back(out, x, dsum=res, dh=(res.window, res.offset + 4)))
        none = N(vr.VR_DT_F32, 0, cols, 1e-5)
        vr.vr_norm(job.comm, none, x, out=out)
        n0 = vr.vr_norm_backward_workspace_bytes(R, none)
        back(out, x, dh=dh, dgain=dg[0], s=none, w=workspace(n0), n=n0)()
        assert not dg[1]().any()  # zeros without rows
        norm(ok, x, gain=gain, residual=res, sum=res, out=out, q8=q8)()
        back(out, x, dsum=res, dh=res, dgain=dg[0])()
        job.assert_no_async_error()
    assert GUARD
