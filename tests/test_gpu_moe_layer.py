"""The few-token mixture-of-experts layer on the GPU against the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import ACT, ACT_EVAL, DT, HALF, STEP, Tensors, check, round_to, workspace
from oracle import layers as L

pytestmark = pytest.mark.gpu


def _data(R, T, E, H, I, dtype, gated, seed):
    rng = np.random.default_rng(seed)
    U = 2 * I if gated else I
    f = lambda *s, k=1.0: round_to(rng.normal(size=s) * k, dtype)  # noqa: E731
    return dict(x=f(R, T, H), w_up=f(R, E // R, U, H, k=H ** -0.5), w_down=f(R, E // R, H, I, k=I ** -0.5),
                residual=f(R, T, H)), f(E, H, k=H ** -0.5)


def _tolerance(d, router, want, idx, weights, act, gated, residual, dtype, H, I, E, K):
    x = d["x"].reshape(-1, H)
    up, down = d["w_up"].reshape(E, -1, H), d["w_down"].reshape(E, H, I)
    tol = np.abs(want) * (HALF[dtype] + 4 * STEP)
    for n in range(x.shape[0]):
        size = np.zeros(H)
        for k in range(K):
            e = idx[n, k]
            if e < 0:
                continue
            z, mag = up[e] @ x[n], np.abs(up[e]) @ np.abs(x[n]) * (H + 4) * STEP
            a, _ = L.activation(z[:I], act)
            ea = 1.2 * mag[:I] + (np.abs(z[:I]) + 1) * ACT_EVAL
            h, eh = (a * z[I:], ea * np.abs(z[I:]) + (np.abs(a) + ea) * mag[I:]) if gated else (a, ea)
            if dtype == "bf16":
                eh = eh + np.abs(h) * 2.0 ** -16  # held as two bf16 parts
            s = np.abs(down[e]) @ (np.abs(h) * (2 * I + 4) * STEP + eh)
            size += weights[n, k] * (s + np.abs(down[e] @ h) * 40 * STEP)
        tol[n] += size
    if residual:
        tol = tol + np.abs(d["residual"].reshape(-1, H)) * 4 * STEP
    return tol


CASES = [  # R, T, E, K, H, I, dtype, act, gated, renorm, residual, off
    (1, 1, 4, 1, 8, 8, "bf16", "silu", True, True, True, 0),
    (1, 1, 64, 8, 256, 128, "bf16", "silu", True, True, True, 0),
    (2, 3, 6, 2, 77, 45, "bf16", "gelu", False, False, False, 1),
    (8, 4, 64, 8, 128, 64, "bf16", "silu", True, True, False, 0),
    (4, 16, 4, 3, 136, 40, "bf16", "relu", True, False, True, 0),
    (1, 64, 5, 5, 64, 96, "bf16", "gelu", True, True, True, 3),
    (1, 2, 1024, 16, 64, 32, "bf16", "silu", False, True, False, 0),
    (3, 5, 9, 4, 50, 33, "f32", "silu", True, True, True, 1),
    (1, 1, 16, 2, 512, 256, "f32", "gelu", False, False, True, 0),
    (2, 32, 8, 8, 68, 36, "f32", "relu", True, False, False, 0),
    (64, 1, 64, 2, 32, 16, "f32", "none", False, True, True, 0),
    (1, 17, 3, 2, 2000, 24, "bf16", "silu", True, True, True, 0),
    (1, 4, 80, 64, 40, 24, "bf16", "silu", True, False, True, 0),
]


@pytest.mark.parametrize("R,T,E,K,H,I,dtype,act,gated,renorm,residual,off", CASES)
def test_moe_layer(R, T, E, K, H, I, dtype, act, gated, renorm, residual, off):
    import torch
    say(f"moe layer R={R} T={T} E={E} K={K} H={H} I={I} {dtype} {act} gated={gated}")
    d, router = _data(R, T, E, H, I, dtype, gated, E + H)
    shape = vr.vrMoeShape(DT[dtype], T, H, I, E, K, ACT[act] | (vr.VR_ACT_GATED if gated else 0),
                          vr.VR_ROUTE_RENORM if renorm else 0)
    need = vr.vr_moe_layer_workspace_bytes(R, shape)
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        s = {k: tn.put(v)[0] for k, v in d.items()}
        out, read = tn.put(shape=(T, H), fill=5.0)
        rt = torch.from_numpy(router).to("cuda").to(tn.tt)
        idx = torch.full((R, T, K), -9, dtype=torch.int32, device="cuda")
        w = torch.full((R, T, K), -9.0, device="cuda")
        ws = workspace(need)
        for _ in range(2):
            vr.vr_moe_layer(job.comm, shape, s["x"], rt, s["w_up"], s["w_down"], out, idx, w,
                            residual=s["residual"] if residual else None, workspace=ws, workspace_bytes=need)
        got = read().reshape(R * T, H)
        want, want_i, want_w = L.moe_layer(d["x"].reshape(-1, H), router, d["w_up"].reshape(E, -1, H),
                                           d["w_down"].reshape(E, H, I), act, gated, K, renorm,
                                           d["residual"].reshape(-1, H) if residual else None)
        assert np.array_equal(idx.cpu().numpy().reshape(R * T, K), want_i)
        check(w.double().cpu().numpy().reshape(R * T, K), want_w, want_w * 4 * STEP + 2.0 ** -140, "weights")
        check(got, want, _tolerance(d, router, want, want_i, want_w, act, gated, residual, dtype, H, I, E, K), "out")
        job.assert_no_async_error()


def test_ties_nan_rows_residual_in_place_and_graph():
    # equal router rows tie to the lowest expert; a NaN token has no experts and keeps its residual
    import torch
    R, T, E, K, H, I = 2, 3, 8, 3, 64, 32
    say("moe layer: ties, NaN token, in place, graph")
    d, router = _data(R, T, E, H, I, "bf16", True, 5)
    router[1:6] = router[0]
    d["x"][1, 2, 7] = np.nan
    shape = vr.vrMoeShape(vr.VR_DT_BF16, T, H, I, E, K, vr.VR_ACT_SILU | vr.VR_ACT_GATED, 0)
    need = vr.vr_moe_layer_workspace_bytes(R, shape)
    with Job(R) as job:
        tn = Tensors(job, "bf16")
        s = {k: tn.put(v)[0] for k, v in d.items()}
        io, read = tn.put(d["residual"])
        out, out_read = tn.put(shape=(T, H))
        rt = torch.from_numpy(router).to("cuda").to(tn.tt)
        idx = torch.zeros((R, T, K), dtype=torch.int32, device="cuda")
        w = torch.zeros((R, T, K), device="cuda")
        ws = workspace(need)

        def run(o, res):
            vr.vr_moe_layer(job.comm, shape, s["x"], rt, s["w_up"], s["w_down"], o, idx, w, residual=res, workspace=ws,
                            workspace_bytes=need)

        run(io, io)
        assert job.async_error()[1] == vr.VR_ASYNC_BAD_VALUE
        got, ids = read(), idx.cpu().numpy()
        assert ids[1, 2].tolist() == [-1] * K and not w[1, 2].any()
        assert np.array_equal(got[1, 2], d["residual"][1, 2])
        x = np.nan_to_num(d["x"].reshape(-1, H))
        want_i = L.route(x @ router.T, K, False)[0].reshape(R, T, K)
        for r in range(R):
            for t in range(T):
                if (r, t) != (1, 2):
                    a = [e for e in ids[r, t] if e < 6]
                    assert a == sorted(a) and (not a or a[0] == 0), ids[r, t]  # the tied ones in order
                    assert set(want_i[r, t]) & {6, 7} == set(ids[r, t]) & {6, 7}
        run(out, s["residual"])
        assert np.array_equal(out_read(), got)
        job.async_error()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            run(out, s["residual"])
        for rep in range(3):
            run(out, None) if rep == 1 else None  # eager work between the replays
            torch.cuda.synchronize()
            graph.replay()
            assert np.array_equal(out_read(), got), rep
        del graph
        job.async_error()


def test_refusals():
    import torch
    say("moe layer refusals")
    R, T, E, K, H, I = 2, 2, 4, 2, 16, 8
    with Job(R) as job:
        tn = Tensors(job, "f32")
        x, up, down, out = (tn.put(shape=v)[0] for v in ((T, H), (E // R, I, H), (E // R, H, I), (T, H)))
        rt = torch.zeros(E, H, device="cuda")
        idx = torch.zeros((R, T, K), dtype=torch.int32, device="cuda")
        w = torch.zeros((R, T, K), device="cuda")
        S = vr.vrMoeShape
        ok = S(0, T, H, I, E, K, 0, 0)
        need = vr.vr_moe_layer_workspace_bytes(R, ok)
        ws = workspace(need)

        def refused(shape, *args, **kw):
            kw = {"workspace": ws, "workspace_bytes": need, **kw}
            with pytest.raises(vr.VrError) as e:
                vr.vr_moe_layer(job.comm, shape, *args, **kw)
            assert e.value.code == vr.VR_ERR_INVALID_ARGUMENT

        for bad in (S(2, T, H, I, E, K, 0, 0), S(0, 33, H, I, E, K, 0, 0), S(0, -1, H, I, E, K, 0, 0),
                    S(0, T, 0, I, E, K, 0, 0), S(0, T, H, 0, E, K, 0, 0), S(0, T, H, I, 5, K, 0, 0),
                    S(0, T, H, I, E, 5, 0, 0), S(0, T, H, I, E, 0, 0, 0), S(0, T, H, I, E, K, 8, 0),
                    S(0, T, H, I, E, K, 0, 2)):
            assert vr.vr_moe_layer_workspace_bytes(R, bad) == 0
            refused(bad, x, rt, up, down, out, idx, w)
        refused(ok, None, rt, up, down, out, idx, w)
        refused(ok, x, None, up, down, out, idx, w)
        refused(ok, x, rt.cpu(), up, down, out, idx, w)
        refused(ok, x, rt, up, down, x, idx, w)
        refused(ok, x, rt, up, down, out, idx, w, workspace_bytes=need - 1)
        refused(ok, x, rt, up, down, out, idx, w, workspace=None)
        refused(ok, x, rt, up, down, out, idx, idx)
        refused(ok, x, rt, up, down, out, None, w)
        vr.vr_moe_layer(job.comm, ok, x, rt, up, down, out, idx, w, workspace=ws, workspace_bytes=need)
        zero = S(0, 0, H, I, E, K, 0, 0)
        vr.vr_moe_layer(job.comm, zero, x, rt, up, down, out, idx, w, workspace=ws,
                        workspace_bytes=max(need, vr.vr_moe_layer_workspace_bytes(R, zero)))
        job.assert_no_async_error()
