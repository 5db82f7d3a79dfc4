"""The linear layer and its gradients on the GPU against the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import ACT, ACT_EVAL, DT, HALF, STEP, Tensors, check, round_to, workspace
from oracle import layers as L

pytestmark = pytest.mark.gpu


def _counts(R, G, rows, seed, used=None):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, max(1, 2 * rows // G), size=(R, G))
    c[rng.random((R, G)) < 0.2] = 0
    for r in range(R):
        while c[r].sum() > (rows if used is None else used):
            c[r, rng.integers(0, G)] //= 2
    return c.astype(np.int32)


def _data(R, rows, G, I, O, dtype, gated, seed):
    rng = np.random.default_rng(seed)
    N = 2 * O if gated else O
    f = lambda *s: round_to(rng.normal(size=s), dtype)  # noqa: E731
    return dict(x=f(R, rows, I), w=round_to(rng.normal(size=(R, G, N, I)) * I ** -0.5, dtype), bias=f(R, G, N),
                residual=f(R, rows, O), dout=f(R, rows, O))


CASES = [  # R, rows, G, I, O, dtype, act, gated, bias, residual, off
    (1, 1, 1, 8, 8, "bf16", "none", False, False, False, 0),
    (1, 1, 1, 256, 512, "bf16", "silu", False, True, True, 0),
    (2, 3, 1, 77, 45, "bf16", "gelu", True, True, True, 1),
    (1, 130, 1, 64, 128, "bf16", "relu", False, True, False, 0),
    (1, 257, 1, 200, 264, "bf16", "silu", True, False, True, 0),
    (1, 300, 1, 1000, 136, "bf16", "gelu", False, True, True, 3),
    (2, 129, 5, 72, 40, "bf16", "silu", True, True, True, 0),
    (4, 70, 16, 33, 17, "bf16", "none", True, False, False, 0),
    (3, 40, 70, 24, 16, "bf16", "gelu", False, True, False, 1),
    (1, 512, 1, 512, 512, "bf16", "none", False, True, False, 0),
    (1, 600, 2, 320, 512, "bf16", "silu", True, True, False, 0),
    (2, 17, 1, 129, 100, "f32", "relu", False, True, True, 1),
    (1, 1, 1, 1, 1, "f32", "none", False, True, True, 0),
    (1, 140, 1, 260, 132, "f32", "silu", True, True, False, 0),
    (2, 90, 6, 50, 36, "f32", "gelu", False, True, True, 0),
    (1, 200, 3, 31, 130, "f32", "none", False, False, False, 1),
    (8, 9, 2, 64, 64, "f32", "silu", True, False, True, 0),
    (1, 16, 1, 4100, 72, "bf16", "none", False, False, True, 0),
    (1, 5, 1, 2048, 33, "f32", "gelu", False, True, False, 0),
    (2, 20, 3, 520, 96, "bf16", "silu", True, True, True, 0),
    (1, 64, 1, 1032, 64, "bf16", "relu", True, True, True, 0),
    # large enough for the widest tiles: forward, dx, dw; contraction lengths of whole steps and with a remainder
    (1, 3700, 1, 200, 3640, "bf16", "silu", False, True, True, 0),
    (1, 3700, 1, 136, 1800, "bf16", "gelu", True, True, False, 0),
    (2, 1900, 3, 3584, 72, "bf16", "none", False, False, False, 0),
    (1, 330, 1, 3648, 3720, "bf16", "relu", False, True, False, 0),
    (2, 150, 2, 1792, 1856, "bf16", "silu", True, False, False, 0),
]


@pytest.mark.parametrize("R,rows,G,I,O,dtype,act,gated,bias,residual,off", CASES)
def test_linear_and_gradients(R, rows, G, I, O, dtype, act, gated, bias, residual, off):
    import torch
    say(f"linear R={R} rows={rows} G={G} I={I} O={O} {dtype} {act} gated={gated} off={off}")
    N = 2 * O if gated else O
    d = _data(R, rows, G, I, O, dtype, gated, rows + I)
    cnt = _counts(R, G, rows, I) if G > 1 else None
    shape = vr.vrLinearShape(DT[dtype], rows, G, I, O, ACT[act] | (vr.VR_ACT_GATED if gated else 0))
    half = HALF[dtype]
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        s = {k: tn.put(v)[0] for k, v in d.items()}
        out, out_read = tn.put(shape=(rows, O), fill=5.0)
        pre, pre_read = tn.put(shape=(rows, N), fill=5.0)
        gr = None if cnt is None else torch.from_numpy(cnt).cuda()
        need = vr.vr_linear_workspace_bytes(R, shape)
        vr.vr_linear(job.comm, shape, s["x"], s["w"], out, bias=s["bias"] if bias else None,
                     residual=s["residual"] if residual else None, preact=pre, group_rows=gr,
                     workspace=workspace(need), workspace_bytes=need)
        got, z_got = out_read(), pre_read()
        job.assert_no_async_error()
        for r in range(R):
            c = None if cnt is None else cnt[r]
            b = d["bias"][r] if bias else None
            want, z = L.linear(d["x"][r], d["w"][r], act, gated, b, d["residual"][r] if residual else None, c)
            used = L.group_ranges([rows] if c is None else c, rows)[-1][1]
            mag = L.linear(np.abs(d["x"][r]), np.abs(d["w"][r]), "none", False, None if b is None else np.abs(b), None, c)[1]
            dz = mag * (I + 4) * STEP  # the sum of I products and the bias
            check(z_got[r, :used], z[:used], (np.abs(z) * half + dz)[:used], "preact")
            a, _ = L.activation(z[:, :O], act)
            da = 1.2 * dz[:, :O] + (np.abs(z[:, :O]) + 1) * ACT_EVAL * (act != "none")  # slopes stay below 1.13
            tol = da * np.abs(z[:, O:]) + (np.abs(a) + da) * dz[:, O:] if gated else da
            tol = tol + np.abs(want) * half + (np.abs(want) + np.abs(d["residual"][r])) * 4 * STEP
            check(got[r, :used], want[:used], tol[:used], "out")
            assert np.all(got[r, used:] == 5.0) and np.all(z_got[r, used:] == 5.0)  # rows of no group

        # the gradients, from the preact that the forward pass left
        dx, dx_read = tn.put(shape=(rows, I), fill=5.0)
        dw, dw_read = tn.put(shape=(G, N, I), fill=5.0)
        db, db_read = tn.put(shape=(G, N), fill=5.0)
        need = vr.vr_linear_backward_workspace_bytes(R, shape)
        plain = act == "none" and not gated
        vr.vr_linear_backward(job.comm, shape, s["dout"], s["x"], s["w"], preact=None if plain else pre, dx=dx, dw=dw,
                              dbias=db, group_rows=gr, workspace=workspace(need), workspace_bytes=need)
        gx, gw, gb = dx_read(), dw_read(), db_read()
        for r in range(R):
            c = None if cnt is None else cnt[r]
            used = L.group_ranges([rows] if c is None else c, rows)[-1][1]
            wx, ww, wb, dzv = L.linear_backward(d["dout"][r], d["x"][r], d["w"][r], None if plain else z_got[r], act, gated, c)
            if plain:
                edz = np.zeros_like(dzv)
                fine = edz
            else:  # the slopes' evaluation, then (bf16) one rounding of dz
                up = np.abs(z_got[r][:, O:]) if gated else 1.0
                fine = np.abs(d["dout"][r]) * up * 4 * ACT_EVAL + np.abs(dzv[:, :O]) * 8 * STEP
                if gated:
                    fine = np.concatenate([fine, np.abs(d["dout"][r]) * (np.abs(z_got[r][:, :O]) + 1) * 4 * ACT_EVAL], 1)
                edz = fine + (np.abs(dzv) * half if dtype == "bf16" else 0.0)
            size = np.abs(dzv) + edz
            tx, tw, _, _ = L.linear_backward(edz + size * (N + 4) * STEP, np.abs(d["x"][r]), np.abs(d["w"][r]), None,
                                             "none", False, c)
            _, tw2, _, _ = L.linear_backward(edz + size * (rows + 4) * STEP, np.abs(d["x"][r]), np.abs(d["w"][r]), None,
                                             "none", False, c)
            _, _, tb, _ = L.linear_backward(fine + size * (rows + 4) * STEP, np.abs(d["x"][r]), np.abs(d["w"][r]), None,
                                            "none", False, c)
            tiny = 2.0 ** -130
            check(gx[r, :used], wx[:used], (tx + np.abs(wx) * half + tiny)[:used], "dx")
            check(gw[r], ww, tw2 + np.abs(ww) * half + tiny, "dw")
            check(gb[r], wb, tb + np.abs(wb) * half + tiny, "dbias")
            assert np.all(gx[r, used:] == 5.0)
        job.assert_no_async_error()


def test_gradient_against_differences():
    import torch
    rows, I, O = 6, 20, 9
    say("linear gradient against differences")
    rng = np.random.default_rng(2)
    d = _data(1, rows, 1, I, O, "f32", True, 4)
    shape = vr.vrLinearShape(vr.VR_DT_F32, rows, 1, I, O, vr.VR_ACT_SILU | vr.VR_ACT_GATED)
    need = vr.vr_linear_backward_workspace_bytes(1, shape)
    eps = 2.0 ** -8
    with Job(1) as job:
        tn = Tensors(job, "f32")

        def run(x, w, b):
            xs, ws, bs = tn.put(x)[0], tn.put(w)[0], tn.put(b)[0]
            out, read = tn.put(shape=(rows, O))
            pre = tn.put(shape=(rows, 2 * O))[0]
            vr.vr_linear(job.comm, shape, xs, ws, out, bias=bs, preact=pre)
            return read(), xs, ws, pre

        _, xs, ws, pre = run(d["x"], d["w"], d["bias"])
        got = {k: tn.put(shape=d[k].shape[1:]) for k in ("x", "w", "bias")}
        vr.vr_linear_backward(job.comm, shape, tn.put(d["dout"])[0], xs, ws, preact=pre, dx=got["x"][0], dw=got["w"][0],
                              dbias=got["bias"][0], workspace=workspace(need), workspace_bytes=need)
        for key in ("x", "w", "bias"):
            v = rng.normal(size=d[key].shape)
            ends = []
            for sgn in (1, -1):
                e = dict(d)
                e[key] = round_to(d[key] + sgn * eps * v, "f32")
                ends.append(run(e["x"], e["w"], e["bias"])[0])
            slope = float(((ends[0] - ends[1]) * d["dout"]).sum()) / (2 * eps)
            have = float((got[key][1]() * v).sum())
            size = float(np.abs(ends[0] * d["dout"]).sum()) + float(np.abs(got[key][1]() * v).sum())
            # the forward's rounding over eps, and the third derivative (below 8 in these units) times eps^2
            assert abs(slope - have) <= size * ((I + 64) * STEP / eps) + 8 * eps ** 2 * float((v ** 2).sum()) ** 1.5, key


def test_group_counts_past_the_rows_and_negative():
    import torch
    say("linear bad group counts")
    rows, G, I, O = 50, 4, 16, 8
    d = _data(1, rows, G, I, O, "f32", False, 9)
    shape = vr.vrLinearShape(vr.VR_DT_F32, rows, G, I, O, vr.VR_ACT_NONE)
    need = vr.vr_linear_backward_workspace_bytes(1, shape)
    for cnt in ([20, -3, 10, 40], [2 ** 31 - 1, 2 ** 31 - 1, 5, 0], [0, 0, 0, -1]):
        with Job(1) as job:
            tn = Tensors(job, "f32")
            s = {k: tn.put(v)[0] for k, v in d.items()}
            out, read = tn.put(shape=(rows, O), fill=5.0)
            dx, _ = tn.put(shape=(rows, I), fill=5.0)
            dw, dwr = tn.put(shape=(G, O, I), fill=5.0)
            db, dbr = tn.put(shape=(G, O), fill=5.0)
            gr = torch.tensor([cnt], dtype=torch.int32, device="cuda")
            vr.vr_linear(job.comm, shape, s["x"], s["w"], out, group_rows=gr)
            assert job.async_error()[1] == vr.VR_ASYNC_CAPACITY
            want, _ = L.linear(d["x"][0], d["w"][0], "none", False, None, None, cnt)
            used = L.group_ranges(cnt, rows)[-1][1]
            got = read()[0]
            check(got[:used], want[:used], 1e-5, "out")
            assert np.all(got[used:] == 5.0)
            vr.vr_linear_backward(job.comm, shape, s["dout"], s["x"], s["w"], dx=dx, dw=dw, dbias=db, group_rows=gr,
                                  workspace=workspace(need), workspace_bytes=need)
            assert job.async_error()[1] == vr.VR_ASYNC_CAPACITY
            _, ww, wb, _ = L.linear_backward(d["dout"][0], d["x"][0], d["w"][0], None, "none", False, cnt)
            check(dwr()[0], ww, 1e-4, "dw")
            check(dbr()[0], wb, 1e-4, "dbias")


def test_residual_in_place_other_stream_and_graph():
    import torch
    say("linear: residual in place, another stream, graph replays")
    rows, I, O = 200, 96, 160
    d = _data(2, rows, 1, I, O, "bf16", False, 12)
    shape = vr.vrLinearShape(vr.VR_DT_BF16, rows, 1, I, O, vr.VR_ACT_GELU)
    need = vr.vr_linear_workspace_bytes(2, shape)
    bneed = vr.vr_linear_backward_workspace_bytes(2, shape)
    with Job(2) as job:
        tn = Tensors(job, "bf16")
        s = {k: tn.put(v)[0] for k, v in d.items()}
        res2, read = tn.put(d["residual"])
        out, out_read = tn.put(shape=(rows, O))
        pre = tn.put(shape=(rows, O))[0]
        dx, dx_read = tn.put(shape=(rows, I))
        dw, dw_read = tn.put(shape=(1, O, I))
        db, db_read = tn.put(shape=(1, O))
        ws, bws = workspace(need), workspace(bneed)

        def both():
            vr.vr_linear(job.comm, shape, s["x"], s["w"], out, bias=s["bias"], residual=s["residual"], preact=pre,
                         workspace=ws, workspace_bytes=need)
            vr.vr_linear_backward(job.comm, shape, s["dout"], s["x"], s["w"], preact=pre, dx=dx, dw=dw, dbias=db,
                                  workspace=bws, workspace_bytes=bneed)

        vr.vr_linear(job.comm, shape, s["x"], s["w"], res2, bias=s["bias"], residual=res2, workspace=ws, workspace_bytes=need)
        both()
        eager = [out_read(), dx_read(), dw_read(), db_read()]
        assert np.array_equal(read(), eager[0])  # in place gives the same
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            both()
        st.synchronize()
        assert all(np.array_equal(a, b()) for a, b in zip(eager, (out_read, dx_read, dw_read, db_read)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            both()
        for rep in range(3):
            for w in (out, dx, dw, db):
                pass
            both() if rep == 1 else None  # eager work between the replays
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(np.array_equal(a, b()) for a, b in zip(eager, (out_read, dx_read, dw_read, db_read))), rep
        del graph


def test_refusals():
    import torch
    say("linear refusals")
    R, rows, I, O = 2, 8, 16, 8
    with Job(R) as job:
        tn = Tensors(job, "f32")
        x, w, out = tn.put(shape=(rows, I))[0], tn.put(shape=(1, O, I))[0], tn.put(shape=(rows, O))[0]
        ok = vr.vrLinearShape(vr.VR_DT_F32, rows, 1, I, O, vr.VR_ACT_NONE)

        def refused(shape, *args, code=vr.VR_ERR_INVALID_ARGUMENT, fn=vr.vr_linear, **kw):
            with pytest.raises(vr.VrError) as e:
                fn(job.comm, shape, *args, **kw)
            assert e.value.code == code

        S = vr.vrLinearShape
        for bad in (S(2, rows, 1, I, O, 0), S(0, -1, 1, I, O, 0), S(0, rows, 0, I, O, 0), S(0, rows, 1025, I, O, 0),
                    S(0, rows, 1, 0, O, 0), S(0, rows, 1, I, 0, 0), S(0, rows, 1, I, O, 4), S(0, rows, 2, I, O, 0),
                    S(0, rows + 64, 1, I, O, 0), S(0, rows, 1, (1 << 20) + 1, O, 0)):
            refused(bad, x, w, out)
        refused(ok, None, w, out)
        refused(ok, x, None, out)
        refused(ok, x, w, None)
        refused(ok, x, w, x)                                   # out over x
        refused(ok, x, w, out, residual=(out.window, out.offset + 4))
        refused(ok, x, w, out, preact=out)
        refused(ok, x, w, (out.window, out.offset + 1))
        refused(ok, x, w, out, group_rows=torch.zeros(R, 1, dtype=torch.int32))  # host memory
        need = vr.vr_linear_backward_workspace_bytes(R, ok)
        assert need > 0 and vr.vr_linear_backward_workspace_bytes(0, ok) == 0
        b = dict(fn=vr.vr_linear_backward)
        ws = workspace(need)
        refused(ok, out, x, w, workspace=ws, workspace_bytes=need, **b)          # nothing wanted
        dx = tn.put(shape=(rows, I))[0]
        refused(ok, out, x, w, dx=dx, workspace=ws, workspace_bytes=need - 1, **b)
        refused(ok, out, x, w, dx=dx, workspace=ws[8:], workspace_bytes=need, **b)
        refused(ok, out, x, w, dx=x, workspace=ws, workspace_bytes=need, **b)
        refused(ok, out, x, None, dx=dx, workspace=ws, workspace_bytes=need, **b)
        act = S(0, rows, 1, I, O, vr.VR_ACT_RELU)
        an = vr.vr_linear_backward_workspace_bytes(R, act)
        refused(act, out, x, w, dx=dx, workspace=workspace(an), workspace_bytes=an, **b)  # no preact
        # a window with VA signal words in the way
        sw, _ = job.window(4096, flags=vr.VR_WIN_STRICT_ORDERING)
        vr.vr_va_signal_reset(job.comm, sw, 0, 64)
        refused(ok, x, w, (sw, 0), code=vr.VR_ERR_INVALID_USAGE)
        vr.vr_linear(job.comm, S(0, 0, 1, I, O, 0), x, w, out)  # no rows
        n0 = vr.vr_linear_workspace_bytes(R, ok)
        vr.vr_linear(job.comm, ok, x, w, out, workspace=workspace(n0), workspace_bytes=n0)
        job.assert_no_async_error()
