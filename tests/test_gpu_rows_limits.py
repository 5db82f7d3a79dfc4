"""The norm, rows in 8 bits, their product and the combine's gradient at large sizes: past the caches, past 2^32 bytes,
more rows than one launch has workgroups, 64 ranks; and the same again and again. Against torch in binary64 on the GPU."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import STEP
from rows_util import pack, q8_window, row_bytes

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def _window(job, shape, dtype, seed=None, scale=1.0):
    """([tensor of each rank], slice); random where seed is given, else 7."""
    import torch
    n = torch.Size(shape).numel()
    h, views = job.window(n * dtype.itemsize, fill=None)
    got = [v.view(dtype).view(shape) for v in views]
    for r, t in enumerate(got):
        if seed is None:
            t.fill_(7)
        else:
            t.copy_(torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed + r), device="cuda") * scale)
    return got, vr.vrSlice(h, 0)


def _scale(m):
    """m / 127 rounded to binary32 once: torch's own division by a number on the GPU is a product with its reciprocal. The
    way by binary64 gives the same as a direct rounding, since 53 >= 2 * 24 + 2."""
    return (m.double() / 127).float()


def _times(m):
    return (127 / m.double()).float().double()


@pytest.mark.parametrize("rows,cols", [(8200, 8192), (70000, 512), (33000, 1024), (40000, 2048)])
def test_calls_larger_than_the_caches(rows, cols):
    import torch
    say(f"norm past the caches: {rows} x {cols} bf16")
    bf = torch.bfloat16
    shape = vr.vrNormShape(vr.VR_DT_BF16, rows, cols, 1e-5)
    with Job(1) as job:
        (x,), xs = _window(job, (rows, cols), bf, 1)
        (res,), rs = _window(job, (rows, cols), bf, 2, 2.0)
        (gain,), gs = _window(job, (cols,), bf, 3)
        (total,), ts = _window(job, (rows, cols), bf)
        (out,), os_ = _window(job, (rows, cols), bf)
        (q8,), qs = _window(job, (rows, row_bytes(cols)), torch.uint8)
        vr.vr_norm(job.comm, shape, xs, gain=gs, residual=rs, sum=ts, out=os_, q8=qs)
        torch.cuda.synchronize()
        assert torch.equal(total, (x.float() + res.float()).to(bf))
        h = total.double()
        root = (h.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        y = h / root * gain.double()
        rel = (cols + 4) * STEP / 2 + 8 * STEP
        assert bool(((out.double() - y).abs() <= y.abs() * (rel + BF) + 2.0 ** -130).all())
        s = q8[:, -4:].contiguous().view(torch.float32).double()
        assert bool(((q8[:, :cols].view(torch.int8).double() * s - y).abs() <= s * (0.5 + 127 * 4 * STEP) + y.abs() * rel).all())
        assert not bool(q8[:, cols:-4].any())
        (dout,), ds = _window(job, (rows, cols), bf, 5)
        (dh,), dhs = _window(job, (rows, cols), bf)
        (dg,), dgs = _window(job, (cols,), bf)
        need = vr.vr_norm_backward_workspace_bytes(1, shape)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        vr.vr_norm_backward(job.comm, shape, ds, ts, gain=gs, dsum=rs, dh=dhs, dgain=dgs, workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        n, w = h / root, dout.double() * gain.double()
        wh = res.double() + (w - n * (w * n).mean(-1, keepdim=True)) / root
        part = (w.abs() * (rel + 8 * STEP) + n.abs() * (w * n).abs().mean(-1, keepdim=True) * ((cols + 4) * STEP + 2 * rel + 8 * STEP)) / root
        assert bool(((dh.double() - wh).abs() <= part + wh.abs() * (BF + 2 * STEP) + 2.0 ** -130).all())
        wg = (dout.double() * n).sum(0)
        assert bool(((dg.double() - wg).abs() <= (dout.double() * n).abs().sum(0) * ((rows + 8) * STEP + rel) + wg.abs() * BF).all())
        job.assert_no_async_error()


@pytest.mark.parametrize("R,rows,cols,dtype", [(8, 2048, 2048, "bf16"), (3, 5462, 1100, "bf16"), (1, 16384, 1023, "f32"),
                                               (8, 4099, 1024, "f32")])
def test_norm_gradients_of_many_rows(R, rows, cols, dtype):
    # dh in dsum's place, also where a row's last 16 bytes are two lanes' (cols no multiple of them)
    import torch
    say(f"norm gradients of many rows: {R} x {rows} x {cols} {dtype}")
    dt, half = (torch.bfloat16, BF) if dtype == "bf16" else (torch.float32, STEP)
    shape = vr.vrNormShape(vr.VR_DT_BF16 if dtype == "bf16" else vr.VR_DT_F32, rows, cols, 1e-5)
    with Job(R) as job:
        h, hs = _window(job, (rows, cols), dt, 1)
        gain, gs = _window(job, (cols,), dt, 20)
        dout, ds = _window(job, (rows, cols), dt, 40)
        dsum, ss = _window(job, (rows, cols), dt, 60)
        dg, dgs = _window(job, (cols,), dt)
        before = [t.double() for t in dsum]
        need = vr.vr_norm_backward_workspace_bytes(R, shape)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        vr.vr_norm_backward(job.comm, shape, ds, hs, gain=gs, dsum=ss, dh=ss, dgain=dgs, workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        rel = (cols + 4) * STEP / 2 + 8 * STEP
        for r in range(R):
            v, d = h[r].double(), dout[r].double()
            root = (v.square().mean(-1, keepdim=True) + 1e-5).sqrt()
            n, w = v / root, d * gain[r].double()
            want = before[r] + (w - n * (w * n).mean(-1, keepdim=True)) / root
            tol = (w.abs() * (rel + 8 * STEP) + n.abs() * (w * n).abs().mean(-1, keepdim=True)
                   * ((cols + 4) * STEP + 2 * rel + 8 * STEP)) / root
            assert bool(((dsum[r].double() - want).abs() <= tol + want.abs() * (half + 2 * STEP) + 2.0 ** -130).all())
            wg = (d * n).sum(0)
            assert bool(((dg[r].double() - wg).abs() <= (d * n).abs().sum(0) * ((rows + 8) * STEP + rel) + wg.abs() * half).all())
        job.assert_no_async_error()


def test_more_rows_than_a_launch_has_workgroups():
    # 2^21 workgroups of a row each, and three rows more; 8.8 GB of values
    import torch
    rows, cols = (1 << 21) + 3, 2104
    say(f"rows in 8 bits: {rows} x {cols}")
    with Job(1) as job:
        h, (view,) = job.window(rows * cols * 2, fill=None)
        x = view.view(torch.bfloat16).view(rows, cols)
        for a in range(0, rows, 1 << 18):
            x[a:a + (1 << 18)].normal_()
        (q8,), qs = _window(job, (rows, row_bytes(cols)), torch.uint8)
        vr.vr_quantize(job.comm, (h, 0), vr.VR_DT_BF16, rows, cols, qs)
        torch.cuda.synchronize()
        for a in range(0, rows, 1 << 18):
            v, q = x[a:a + (1 << 18)].float(), q8[a:a + (1 << 18)]
            m = v.abs().amax(-1, keepdim=True)
            assert torch.equal(q[:, -4:].contiguous().view(torch.float32), _scale(m))
            assert torch.equal(q[:, :cols].view(torch.int8), torch.round(v.double() * _times(m)).to(torch.int8))
            assert not bool(q[:, cols:-4].any())
        x.fill_(7)
        vr.vr_dequantize(job.comm, qs, vr.VR_DT_BF16, rows, cols, (h, 0))
        torch.cuda.synchronize()
        for a in range(0, rows, 1 << 18):
            q = q8[a:a + (1 << 18)]
            want = q[:, :cols].view(torch.int8).float() * q[:, -4:].contiguous().view(torch.float32)
            assert torch.equal(x[a:a + (1 << 18)], want.to(torch.bfloat16))
        job.assert_no_async_error()


def test_narrow_rows_by_the_million():
    import torch
    rows, cols = 5000001, 12
    say(f"rows in 8 bits: {rows} x {cols}")
    with Job(1) as job:
        (x,), xs = _window(job, (rows, cols), torch.float32, 1)
        (q8,), qs = _window(job, (rows, 128), torch.uint8)
        vr.vr_quantize(job.comm, xs, vr.VR_DT_F32, rows, cols, qs)
        torch.cuda.synchronize()
        m = x.abs().amax(-1, keepdim=True)
        assert torch.equal(q8[:, -4:].contiguous().view(torch.float32), _scale(m))
        assert torch.equal(q8[:, :cols].view(torch.int8), torch.round(x.double() * _times(m)).to(torch.int8))
        job.assert_no_async_error()


def test_combine_gradient_far_into_a_window():
    import torch
    R, T, E, K, cols, cap = 2, 5, 4, 3, 30000, 80000  # rows of 60000 bytes: 4.8 GB a rank
    say("combine backward: offsets past 32 bits")
    gen = torch.Generator(device="cuda").manual_seed(1)
    bf = torch.bfloat16
    with Job(R) as job:
        dout, ds = _window(job, (T, cols), bf, 1)
        y, ys = _window(job, (cap, cols), bf)
        dy, dys = _window(job, (cap, cols), bf)
        topk = torch.randint(0, E, (R, T, K), generator=gen, device="cuda", dtype=torch.int32)
        pos = (cap - 1 - torch.randperm(R * T * K, generator=gen, device="cuda") * 2000).view(R, T, K).to(torch.int32)
        assert int(pos.min()) * cols * 2 < 1 << 32 < int(pos.max()) * cols * 2
        w = torch.randn(R, T, K, generator=gen, device="cuda")
        dw = torch.empty(R, T, K, device="cuda")
        for at in np.ndindex(R, T, K):
            y[int(topk[at]) // 2][int(pos[at])].copy_(torch.randn(cols, generator=gen, device="cuda"))
        vr.vr_combine_backward(job.comm, ds, ys, cap, cols * 2, vr.VR_DT_BF16, topk, w, pos, T, K, E, dy=dys, dweights=dw)
        torch.cuda.synchronize()
        for at in np.ndindex(R, T, K):
            d, p, src = int(topk[at]) // 2, int(pos[at]), dout[at[0]][at[1]].double()
            want = src * w[at].double()
            assert bool(((dy[d][p].double() - want).abs() <= want.abs() * (BF + STEP)).all())
            dot = src * y[d][p].double()
            assert abs(float(dw[at]) - float(dot.sum())) <= float(dot.abs().sum()) * (cols + 8) * STEP
            dy[d][p] = 7
        assert all(bool((t == 7).all()) for t in dy)  # nothing else was written
        job.assert_no_async_error()


def test_64_ranks():
    import torch
    say("64 ranks")
    R, rows, cols, G, O = 64, 5, 72, 2, 40  # noqa: E741
    gen = torch.Generator(device="cuda").manual_seed(1)
    with Job(R) as job:
        x, xs = _window(job, (rows, cols), torch.float32, 1)
        w, ws_ = _window(job, (G * O, cols), torch.float32, 100, cols ** -0.5)
        x8, x8s = _window(job, (rows, row_bytes(cols)), torch.uint8)
        w8, w8s = _window(job, (G * O, row_bytes(cols)), torch.uint8)
        out, os_ = _window(job, (rows, O), torch.float32)
        norm = vr.vrNormShape(0, rows, cols, 1e-5)
        vr.vr_norm(job.comm, norm, xs, q8=x8s)
        vr.vr_quantize(job.comm, ws_, 0, G * O, cols, w8s)
        counts = torch.tensor([[2, 2]] * R, dtype=torch.int32, device="cuda")
        vr.vr_linear_q8(job.comm, vr.vrLinearShape(0, rows, G, cols, O, 0), x8s, w8s, os_, group_rows=counts)
        need = vr.vr_norm_backward_workspace_bytes(R, norm)
        room = torch.empty(need, dtype=torch.uint8, device="cuda")
        dg, dgs = _window(job, (cols,), torch.float32)
        vr.vr_norm_backward(job.comm, norm, xs, xs, dgain=dgs, workspace=room, workspace_bytes=need)
        T, K, E = 3, 4, 128
        topk = torch.randint(0, E, (R, T, K), generator=gen, device="cuda", dtype=torch.int32)
        pos = torch.full((R, T, K), -1, dtype=torch.int32, device="cuda")
        used = [0] * R
        for at in np.ndindex(R, T, K):
            d = int(topk[at]) // 2
            if used[d] < rows:
                pos[at], used[d] = used[d], used[d] + 1
        dy, dys = _window(job, (rows, cols), torch.float32)
        weights, dw = torch.rand(R, T, K, generator=gen, device="cuda"), torch.empty(R, T, K, device="cuda")
        vr.vr_combine_backward(job.comm, xs, xs, rows, cols * 4, 0, topk, weights, pos, T, K, E, dy=dys, dweights=dw)
        torch.cuda.synchronize()
        for r in range(R):
            h = x[r].double()
            n = h / (h.square().mean(-1, keepdim=True) + 1e-5).sqrt()
            v8, s8 = x8[r][:, :cols].view(torch.int8).double(), x8[r][:, -4:].contiguous().view(torch.float32).double()
            assert bool(((v8 * s8 - n).abs() <= s8 * 0.5001 + 1e-5).all())
            ww = w8[r][:, :cols].view(torch.int8).double() * w8[r][:, -4:].contiguous().view(torch.float32).double()
            for g in range(G):
                want = (v8 * s8)[2 * g:2 * g + 2] @ ww[g * O:(g + 1) * O].T
                assert bool(((out[r][2 * g:2 * g + 2].double() - want).abs() <= 1e-5).all())
            assert bool((out[r][4] == 7).all())
            assert bool(((dg[r].double() - (h * n).sum(0)).abs() <= 1e-4 * (h * n).abs().sum(0)).all())
        for at in np.ndindex(R, T, K):
            if int(pos[at]) < 0:
                assert float(dw[at]) == 0
                continue
            d, p = int(topk[at]) // 2, int(pos[at])
            src = x[at[0]][at[1]].double()
            assert bool(((dy[d][p].double() - src * weights[at].double()).abs() <= src.abs() * 2 * STEP).all())
            dot = src * x[d][p].double()
            assert abs(float(dw[at]) - float(dot.sum())) <= float(dot.abs().sum()) * (cols + 8) * STEP
        job.assert_no_async_error()


@pytest.mark.parametrize("R,rows,G,I,O,act", [(8, 6000, 8, 512, 512, vr.VR_ACT_SILU | vr.VR_ACT_GATED), (1, 8192, 1, 300, 4096, vr.VR_ACT_NONE),
                                              (3, 5000, 40, 1100, 700, vr.VR_ACT_RELU)])
def test_tile_after_tile_gives_the_same_every_time(R, rows, G, I, O, act):  # noqa: E741
    # workgroups that take many tiles, whole and ragged ones, other ranks' groups: their loads run ahead of their stores
    import torch
    say(f"linear q8 again and again: R={R} rows={rows} G={G} I={I} O={O}")
    rng = np.random.default_rng(1)
    N = 2 * O if act & vr.VR_ACT_GATED else O
    data = lambda *s: pack(rng.integers(-127, 128, size=(R, *s, I), dtype=np.int8), rng.uniform(0.5, 1.5, size=(R, *s)).astype(np.float32) / 400)  # noqa: E731
    with Job(R) as job:
        px, pw = data(rows), data(G, N)
        x, w = q8_window(job, px.shape[1:], px)[0], q8_window(job, pw.shape[1:], pw)[0]
        out, os_ = _window(job, (rows, O), torch.bfloat16)
        counts = None
        if G > 1:
            share = rng.uniform(0, 1, size=(R, G)) * (rng.random((R, G)) > 0.2)
            counts = torch.from_numpy(np.floor(share / share.sum(1, keepdims=True) * (rows - 100)).astype(np.int32)).cuda()
        shape = vr.vrLinearShape(vr.VR_DT_BF16, rows, G, I, O, act)
        run = lambda: vr.vr_linear_q8(job.comm, shape, x, w, os_, group_rows=counts)  # noqa: E731
        run()
        first = [t.clone() for t in out]
        wide = lambda p: torch.from_numpy(p[..., :I].view(np.int8)).cuda().double() * torch.from_numpy(np.ascontiguousarray(p[..., -4:]).view(np.float32)).cuda().double()  # noqa: E731
        for r in range(R):
            xd, at = wide(px[r]), 0
            for g, n in enumerate([rows] if counts is None else counts[r].tolist()):
                z = xd[at:at + n] @ wide(pw[r, g]).T
                want = torch.nn.functional.silu(z[:, :O]) * z[:, O:] if N > O else z.relu() if act else z
                # a product's three roundings, an activation in bf16's arithmetic (2^-12 of it), the output's
                assert bool(((first[r][at:at + n].double() - want).abs() <= want.abs() * (BF + 2.0 ** -10) + 1e-5).all()), (r, g)
                at += n
            assert bool((first[r][at:] == 7).all())
        for rep in range(15):
            for t in out:
                t.fill_(9)
            run()
            for r in range(R):
                used = rows if counts is None else int(counts[r].sum())
                assert torch.equal(out[r][:used], first[r][:used]), rep
                assert bool((out[r][used:] == 9).all())
        job.assert_no_async_error()
