"""The combine's gradient on the GPU against the binary64 definition, at the places that vr_dispatch gives the rows."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors, check, round_to
from oracle import layers as L
from rows_util import refused

pytestmark = pytest.mark.gpu


def _routing(rng, R, T, E, K, empty):
    """topk [R][T][K] (an expert may come twice), and the dispatch's places: by expert, source, token, entry."""
    topk = rng.integers(0, E, size=(R, T, K)).astype(np.int32)
    topk[rng.random((R, T, K)) < empty] = -1
    per, pos, n = E // R, np.full((R, T, K), -1, np.int32), [0] * R
    for e in range(E):
        for at in np.argwhere(topk == e):
            pos[tuple(at)] = n[e // per]
            n[e // per] += 1
    return topk, pos, max(n)


CASES = [  # R, T, E, K, cols, dtype, empty, off
    (1, 1, 1, 1, 1, "f32", 0.0, 0), (1, 1, 8, 4, 256, "bf16", 0.0, 0), (2, 37, 8, 3, 77, "f32", 0.2, 1),
    (3, 37, 72, 5, 77, "bf16", 0.2, 1), (4, 20, 16, 8, 256, "bf16", 0.0, 0), (8, 65, 64, 8, 256, "bf16", 0.1, 0),
    (1, 100, 16, 2, 8, "bf16", 0.5, 0), (2, 33, 4, 9, 64, "f32", 0.0, 0), (1, 9, 4, 64, 40, "bf16", 0.3, 0),
    (2, 17, 6, 17, 130, "f32", 0.1, 3), (4, 11, 8, 4, 2048, "bf16", 0.0, 0), (1, 5, 8, 8, 4100, "f32", 0.0, 0),
    (2, 6, 8, 2, 1001, "bf16", 0.0, 1), (1, 40, 1024, 8, 512, "bf16", 0.0, 0), (2, 5, 4, 3, 16, "bf16", 1.0, 0),
]


@pytest.mark.parametrize("R,T,E,K,cols,dtype,empty,off", CASES)
def test_combine_backward(R, T, E, K, cols, dtype, empty, off):
    import torch
    say(f"combine backward R={R} T={T} E={E} K={K} cols={cols} {dtype} empty={empty} off={off}")
    rng = np.random.default_rng(T * K + cols)
    topk, pos, most = _routing(rng, R, T, E, K, empty)
    cap = max(1, most - most // 8) + 2  # some rows fell past the capacity, or two are nobody's
    pos[pos >= cap] = -1
    dout, y = round_to(rng.normal(size=(R, T, cols)), dtype), round_to(rng.normal(size=(R, cap, cols)), dtype)
    w = rng.normal(size=(R, T, K)).astype(np.float32)
    want, want_w = L.combine_backward(dout, y, np.where(topk < 0, -1, topk // (E // R)), pos, w)
    rb = cols * (4 if dtype == "f32" else 2)
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        d, ys = tn.put(dout)[0], tn.put(y)[0]
        dy, read = tn.put(shape=(cap, cols), fill=5.0)
        gt, gp, gw = (torch.from_numpy(v).cuda() for v in (topk, pos, w))
        dw = torch.full((R * T * K + 2,), 7.0, device="cuda")
        call = lambda **k: vr.vr_combine_backward(job.comm, d, ys, cap, rb, DT[dtype], gt, gw, gp, T, K, E, **k)  # noqa: E731
        call(dy=dy, dweights=dw[1:-1])
        got, got_w = read(), dw.cpu().double().numpy()
        job.assert_no_async_error()
        assert got_w[0] == got_w[-1] == 7.0
        for r in range(R):
            for p in range(cap):
                if (r, p) in want:
                    check(got[r, p], want[r, p], np.abs(want[r, p]) * (HALF[dtype] + STEP) + 2.0 ** -130, "dy")
                else:
                    assert np.all(got[r, p] == 5.0)  # a row that no entry names
        mag = L.combine_backward(np.abs(dout), np.abs(y), np.where(topk < 0, -1, topk // (E // R)), pos, w)[1]
        check(got_w[1:-1].reshape(R, T, K), want_w, mag * (cols + 8) * STEP, "dweights")
        # either alone gives the same; again the same
        dy2, read2 = tn.put(shape=(cap, cols), fill=5.0)
        call(dy=dy2)
        assert np.array_equal(read2(), got)
        dw2 = torch.full((R * T * K,), 7.0, device="cuda")
        call(dweights=dw2)
        assert torch.equal(dw2, dw[1:-1])
        vr.vr_combine_backward(job.comm, d, None, cap, rb, DT[dtype], gt, gw, gp, T, K, E, dy=dy2)
        assert np.array_equal(read2(), got)


@pytest.mark.parametrize("dtype,cols", [("bf16", 96), ("f32", 50)])
def test_against_differences_of_the_combine(dtype, cols):
    # the forward's own outputs at weights and rows a step apart: linear in each, so differences are exact but for rounding
    import torch
    say(f"combine backward against the combine's differences, {dtype}")
    R, T, E, K = 2, 9, 8, 3
    rng = np.random.default_rng(6)
    topk, pos, cap = _routing(rng, R, T, E, K, 0.1)
    dout, y, v = (round_to(rng.normal(size=s), dtype) for s in ((R, T, cols), (R, cap, cols), (R, cap, cols)))
    w, u = rng.normal(size=(R, T, K)).astype(np.float32), rng.normal(size=(R, T, K)).astype(np.float32)
    rb = cols * (4 if dtype == "f32" else 2)
    with Job(R) as job:
        tn = Tensors(job, dtype)
        gt, gp = torch.from_numpy(topk).cuda(), torch.from_numpy(pos).cuda()

        def forward(y, w):
            out, read = tn.put(shape=(T, cols))
            src = tn.put(y)[0]
            vr.vr_combine(job.comm, src.window, src.offset, cap, rb, DT[dtype], gt, torch.from_numpy(w).cuda(), gp, T, K, E,
                          out.window, out.offset, 0)
            return read()

        dy, read = tn.put(shape=(cap, cols))
        dw = torch.empty(R, T, K, device="cuda")
        vr.vr_combine_backward(job.comm, tn.put(dout)[0], tn.put(y)[0], cap, rb, DT[dtype], gt, torch.from_numpy(w).cuda(), gp, T, K,
                               E, dy=dy, dweights=dw)
        base = forward(y, w)
        for name, moved, have in (("y", forward(round_to(y + v, dtype), w), (read() * (round_to(y + v, dtype) - y)).sum()),
                                  ("weights", forward(y, w + u), (dw.cpu().double().numpy() * ((w + u).astype(np.float64) - w)).sum())):
            slope = ((moved - base) * dout).sum()
            size = ((np.abs(moved) + np.abs(base)) * np.abs(dout)).sum() + np.abs(read() * (np.abs(y) + np.abs(v))).sum()
            assert abs(slope - have) <= size * (HALF[dtype] + (K + cols) * STEP), name
        job.assert_no_async_error()


def test_ids_and_places_out_of_range_are_skipped():
    import torch
    say("combine backward: bad ids and places")
    R, T, E, K, cols, cap = 2, 4, 4, 3, 24, 10
    rng = np.random.default_rng(6)
    dout, y = round_to(rng.normal(size=(R, T, cols)), "f32"), round_to(rng.normal(size=(R, cap, cols)), "f32")
    topk, pos = np.full((R, T, K), -1, np.int32), np.full((R, T, K), -1, np.int32)
    topk[0, 0], pos[0, 0] = [0, 4, 3], [0, 1, 2]         # expert 4 of 4
    topk[0, 1], pos[0, 1] = [1, 2, -2], [3, 4, 5]        # expert -2
    topk[1, 2], pos[1, 2] = [0, 1, 3], [cap, -7, cap - 1]  # places past the rows and negative
    w = np.ones((R, T, K), np.float32)
    good_t, good_p = np.where((topk < 0) | (topk >= E) | (pos < 0) | (pos >= cap), -1, topk), pos
    want, want_w = L.combine_backward(dout, y, np.where(good_t < 0, -1, good_t // 2), good_p, w)
    assert len(want) == 5
    with Job(R) as job:
        tn = Tensors(job, "f32")
        dy, read = tn.put(shape=(cap, cols), fill=5.0)
        dw = torch.full((R, T, K), 7.0, device="cuda")
        vr.vr_combine_backward(job.comm, tn.put(dout)[0], tn.put(y)[0], cap, cols * 4, 0, torch.from_numpy(topk).cuda(),
                               torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda(), T, K, E, dy=dy, dweights=dw)
        assert job.async_error()[1] == vr.VR_ASYNC_BAD_EXPERT | vr.VR_ASYNC_CAPACITY
        got = read()
        for r, p in np.ndindex(R, cap):
            assert np.array_equal(got[r, p], want[r, p]) if (r, p) in want else np.all(got[r, p] == 5.0)
        check(dw.cpu().double().numpy(), want_w, 1e-4, "dweights")
        assert not dw.cpu().numpy()[want_w == 0].any()


def test_no_tokens_and_refusals():
    import torch
    say("combine backward: no tokens, refusals")
    R, T, E, K, cols, cap = 2, 4, 4, 3, 24, 10
    rb = cols * 4
    with Job(R) as job:
        tn = Tensors(job, "f32")
        d, y, dy = tn.put(shape=(T, cols))[0], tn.put(shape=(cap, cols))[0], tn.put(shape=(cap, cols))[0]
        i32 = dict(dtype=torch.int32, device="cuda")
        topk, pos = torch.full((R, T, K), -1, **i32), torch.full((R, T, K), -1, **i32)
        w, dw = torch.zeros(R, T, K, device="cuda"), torch.zeros(R, T, K, device="cuda")

        def call(d=d, y=y, cap=cap, rb=rb, dt=0, topk=topk, w=w, pos=pos, T=T, K=K, E=E, **k):
            return lambda: vr.vr_combine_backward(job.comm, d, y, cap, rb, dt, topk, w, pos, T, K, E, **(k or dict(dy=dy, dweights=dw)))

        refused(call(dt=2))
        refused(call(T=-1))
        refused(call(T=65536))
        refused(call(K=0))
        refused(call(K=65))
        refused(call(E=3))
        refused(call(E=1026))
        refused(call(rb=0))
        refused(call(rb=rb + 2))
        refused(call(rb=rb * 16))
        refused(call(cap=cap + 64))
        refused(call(d=None))
        refused(call(y=None))                        # dweights need it
        refused(call(dy=None, dweights=None))
        refused(call(dy=y, dweights=dw))
        refused(call(dy=d, dweights=dw))
        refused(call(dy=(dy.window, dy.offset + 2)))
        refused(call(topk=topk.cpu()))
        refused(call(w=None))
        refused(call(pos=None))
        refused(call(dweights=w))
        refused(call(dweights=w.cpu()))
        refused(call(dweights=dw.data_ptr() + 2))
        sw, _ = job.window(4096, flags=vr.VR_WIN_STRICT_ORDERING)
        vr.vr_va_signal_reset(job.comm, sw, 0, 64)
        refused(call(dy=(sw, 0)), vr.VR_ERR_INVALID_USAGE)
        call(T=0, topk=None, w=None, pos=None)()
        call()()
        job.assert_no_async_error()
