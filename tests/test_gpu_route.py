"""The router and its gradient on the GPU against the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors, check, round_to
from oracle import layers as L

pytestmark = pytest.mark.gpu


def _logits(R, T, E, dtype, seed, masked=0, levels=None):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(R, T, E)) * 2
    if levels:
        x = rng.integers(0, levels, size=(R, T, E)).astype(np.float64)  # many ties
    x = round_to(x, dtype)
    if masked:
        order = rng.random((R, T, E)).argsort(-1)
        x[order < masked] = -np.inf
    return x


def _weight_tol(x, w):
    """Relative: the arguments' rounding (half a step of |x - max|), exp within 4 steps, a sum of at most 16 + 6
    additions, one division."""
    fin = np.where(np.isfinite(x), x, 0.0)
    return w * (np.abs(fin).max() * 2 + 32) * STEP + 2.0 ** -140


CASES = [  # R, T, E, K, dtype, renorm, masked, levels, off
    (1, 1, 64, 4, "bf16", True, 0, None, 0), (1, 1, 1, 1, "f32", False, 0, None, 0), (3, 67, 72, 5, "f32", True, 9, None, 0),
    (2, 33, 256, 8, "bf16", False, 0, None, 0), (4, 65, 128, 64, "f32", False, 70, None, 1),
    (8, 9, 1024, 16, "bf16", True, 0, None, 3), (1, 130, 513, 7, "f32", True, 0, 4, 1), (2, 50, 96, 8, "bf16", False, 90, 3, 5),
    (5, 11, 10, 10, "f32", True, 0, 2, 0), (8, 300, 256, 8, "f32", True, 0, None, 0), (1, 257, 257, 16, "bf16", False, 255, None, 1),
]


@pytest.mark.parametrize("R,T,E,K,dtype,renorm,masked,levels,off", CASES)
def test_route_and_gradient(R, T, E, K, dtype, renorm, masked, levels, off):
    import torch
    say(f"route R={R} T={T} E={E} K={K} {dtype} renorm={renorm} masked={masked} off={off}")
    x = _logits(R, T, E, dtype, R * T + E, masked, levels)
    flags = vr.VR_ROUTE_RENORM if renorm else 0
    want_i, want_w = L.route(x, K, renorm)
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        xs, _ = tn.put(x)
        ds, dread = tn.put(shape=(T, E), fill=3.0)
        idx = torch.full((R, T, K), -9, dtype=torch.int32, device="cuda")
        w = torch.full((R, T, K), -9.0, device="cuda")
        vr.vr_route(job.comm, xs, DT[dtype], T, K, E, idx, w, flags)
        got_w = w.double().cpu().numpy()
        assert np.array_equal(idx.cpu().numpy(), want_i)
        check(got_w, want_w, _weight_tol(x, want_w), "weights")
        dw = np.random.default_rng(1).normal(size=(R, T, K)).astype(np.float32)
        vr.vr_route_backward(job.comm, None if renorm else xs, DT[dtype], T, K, E, idx, w,
                             torch.from_numpy(dw).cuda(), ds, flags)
        want = L.route_backward(x, want_i, got_w, dw, renorm)
        # p and the difference dw - m (K products summed) in binary32, one rounding to the type
        m = x.max(-1, keepdims=True)
        full = np.where(np.isfinite(x), np.exp(x - np.where(np.isfinite(m), m, 0.0)), 0.0)
        full = full / np.maximum(full.sum(-1, keepdims=True), 2.0 ** -100)
        scale = np.abs(dw).max() * 2
        fin = np.where(np.isfinite(x), x, 0.0)
        rel = (np.abs(fin).max() * 2 + 32 + K) * STEP
        base = full if not renorm else np.where(want != 0, 1.0, 0.0)
        check(dread(), want, np.abs(want) * HALF[dtype] + base * scale * rel + 2.0 ** -130, "dlogits")
        job.assert_no_async_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_masks_leave_empty(dtype):
    # all masked by -inf; all at the type's lowest value (a uniform row); one left; NaN and +inf in places
    import torch
    R, T, E, K = 2, 5, 20, 3
    say(f"route masks {dtype}")
    low = float(torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min)
    x = np.zeros((R, T, E))
    x[:, 0] = -np.inf
    x[:, 1] = low
    x[:, 2] = -np.inf
    x[:, 2, 11] = -3.0
    x[:, 3] = np.where(np.arange(E) % 2, low, 1.0)
    x[:, 4, 3] = np.nan
    x[:, 4, 4] = np.inf
    with Job(R) as job:
        tn = Tensors(job, dtype)
        xs, _ = tn.put(x)
        ds, dread = tn.put(shape=(T, E))
        for flags in (0, vr.VR_ROUTE_RENORM):
            idx = torch.zeros((R, T, K), dtype=torch.int32, device="cuda")
            w = torch.zeros((R, T, K), device="cuda")
            vr.vr_route(job.comm, xs, DT[dtype], T, K, E, idx, w, flags)
            code, bits = job.async_error()
            assert code == vr.VR_ERR_DEVICE_CHECK and bits == vr.VR_ASYNC_BAD_VALUE
            want_i, want_w = L.route(x, K, bool(flags))
            assert np.array_equal(idx.cpu().numpy(), want_i)
            assert idx[0].tolist() == [[-1, -1, -1], [0, 1, 2], [11, -1, -1], [0, 2, 4], [0, 1, 2]]
            check(w.double().cpu().numpy(), want_w, want_w * 40 * STEP, "weights")
            vr.vr_route_backward(job.comm, xs, DT[dtype], T, K, E, idx, w, torch.ones((R, T, K), device="cuda"), ds, flags)
            got = dread()
            assert np.isfinite(got).all() and not got[:, 0].any() and not got[:, 2].any()
            job.async_error()


def test_gradient_against_differences():
    # the directional derivative of sum(weights * dw), central differences of the GPU's own forward
    import torch
    R, T, E, K = 1, 8, 64, 6
    say("route gradient against differences")
    rng = np.random.default_rng(8)
    x = rng.permutation(R * T * E).reshape(R, T, E) / 100.0  # gaps of 0.01 keep the choice fixed
    x = round_to(x - x.mean(-1, keepdims=True), "f32")
    v, dw = rng.normal(size=x.shape), rng.normal(size=(R, T, K)).astype(np.float32)
    eps = 2.0 ** -10
    for flags in (0, vr.VR_ROUTE_RENORM):
        with Job(R) as job:
            tn = Tensors(job, "f32")
            out = []
            for step in (eps, -eps):
                s, _ = tn.put(round_to(x + step * v, "f32"))
                idx = torch.zeros((R, T, K), dtype=torch.int32, device="cuda")
                w = torch.zeros((R, T, K), device="cuda")
                vr.vr_route(job.comm, s, vr.VR_DT_F32, T, K, E, idx, w, flags)
                out.append((idx.cpu().numpy(), w.double().cpu().numpy()))
            assert np.array_equal(out[0][0], out[1][0])
            s, _ = tn.put(x)
            ds, dread = tn.put(shape=(T, E))
            vr.vr_route(job.comm, s, vr.VR_DT_F32, T, K, E, idx, w, flags)
            vr.vr_route_backward(job.comm, s, vr.VR_DT_F32, T, K, E, idx, w, torch.from_numpy(dw).cuda(), ds, flags)
            slope = ((out[0][1] - out[1][1]) * dw).sum((-1, -2)) / (2 * eps)
            got = (dread() * v).sum((-1, -2))
            # weights' error 64 steps over 2 eps, the inputs' rounding over eps, the third derivative eps^2
            tol = T * K * np.abs(dw).max() * (64 * STEP / eps + 2.0 ** -20 / eps * 0.25) + T * K * 100 * eps ** 2
            assert np.all(np.abs(slope - got) <= tol), (slope, got, tol)


def test_gradient_skips_bad_ids_and_may_write_over_the_logits():
    import torch
    R, T, E, K = 2, 3, 12, 2
    say("route backward bad ids, in place")
    x = _logits(R, T, E, "f32", 3)
    idx, w = L.route(x, K, False)
    dw = np.ones((R, T, K), np.float32)
    bad = idx.copy()
    bad[0, 0, 0], bad[1, 2, 1] = E, -2
    with Job(R) as job:
        xs, read = Tensors(job, "f32").put(x)
        vr.vr_route_backward(job.comm, xs, vr.VR_DT_F32, T, K, E, torch.from_numpy(bad).cuda(),
                             torch.from_numpy(w.astype(np.float32)).cuda(), torch.from_numpy(dw).cuda(), xs)
        code, bits = job.async_error()
        assert code == vr.VR_ERR_DEVICE_CHECK and bits == vr.VR_ASYNC_BAD_EXPERT
        skip = np.where((bad < 0) | (bad >= E), -1, bad)
        want = L.route_backward(x, skip, w.astype(np.float32), dw, False)
        check(read(), want, np.abs(want) * 2.0 ** -24 + 80 * STEP, "dlogits")


def test_refusals():
    import torch
    R, T, E, K = 2, 4, 8, 2
    say("route refusals")
    with Job(R) as job:
        xs, _ = Tensors(job, "f32").put(shape=(T, E))
        idx = torch.zeros((R, T, K), dtype=torch.int32, device="cuda")
        w = torch.zeros((R, T, K), device="cuda")
        f = vr.VR_DT_F32

        def refused(*args, fn=vr.vr_route):
            with pytest.raises(vr.VrError) as e:
                fn(job.comm, *args)
            assert e.value.code == vr.VR_ERR_INVALID_ARGUMENT

        refused(xs, 2, T, K, E, idx, w)
        refused(xs, f, T, 0, E, idx, w)
        refused(xs, f, T, 65, E, idx, w)
        refused(xs, f, T, K, 7, idx, w)
        refused(xs, f, T, K, 1026, idx, w)
        refused(xs, f, -1, K, E, idx, w)
        refused(xs, f, 4096, K, E, idx, w)  # past the window
        refused(None, f, T, K, E, idx, w)
        refused((xs.window, 2), f, T, K, E, idx, w)  # misaligned
        refused(xs, f, T, K, E, idx.cpu(), w)
        refused(xs, f, T, K, E, idx, idx)
        refused(xs, f, T, K, E, idx, w, 2)
        refused(None, f, T, K, E, idx, w, w, xs, fn=vr.vr_route_backward)
        refused(xs, f, T, K, E, idx, w, w, None, fn=vr.vr_route_backward)
        refused(xs, f, T, K, E, idx, w, w, (xs.window, xs.offset + 4), fn=vr.vr_route_backward)
        vr.vr_route(job.comm, xs, f, 0, K, E, None, None)  # no tokens
        vr.vr_route(job.comm, xs, f, T, K, E, idx, w)
        job.assert_no_async_error()
