"""The matrix product of rows in 8 bits on the GPU against the binary64 definition."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import ACT, ACT_EVAL, DT, HALF, STEP, Tensors, check, round_to
from oracle import layers as L
from rows_util import pack, q8_window, refused, row_bytes

pytestmark = pytest.mark.gpu


def _counts(R, G, rows, seed):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, max(1, 2 * rows // G), size=(R, G))
    c[rng.random((R, G)) < 0.2] = 0
    for r in range(R):
        while c[r].sum() > rows:
            c[r, rng.integers(0, G)] //= 2
    return c.astype(np.int32)


def _rows8(rng, *shape):
    """Values -127..127 and scales of about 1 / 40."""
    v = np.clip(np.rint(rng.normal(size=shape) * 40), -127, 127).astype(np.int8)
    return v, (rng.uniform(0.5, 1.5, size=shape[:-1]) / 40).astype(np.float32)


CASES = [  # R, rows, G, I, O, dtype, act, gated, bias, residual, off (bytes of the q8 rows / 4, elements of the others)
    (1, 1, 1, 1, 1, "f32", "none", False, False, False, 0),
    (1, 1, 1, 4096, 512, "bf16", "silu", False, True, True, 0),
    (2, 3, 1, 77, 45, "bf16", "gelu", True, True, True, 1),
    (1, 16, 1, 124, 33, "f32", "relu", False, True, True, 0),
    (1, 32, 1, 125, 48, "f32", "silu", True, False, False, 3),
    (1, 33, 1, 128, 64, "bf16", "relu", False, True, False, 0),
    (1, 130, 1, 640, 128, "bf16", "none", False, True, False, 0),
    (1, 257, 1, 200, 264, "bf16", "silu", True, False, True, 0),
    (1, 300, 1, 1000, 136, "bf16", "gelu", False, True, True, 3),
    (2, 129, 5, 72, 40, "bf16", "silu", True, True, True, 0),
    (4, 70, 16, 33, 17, "bf16", "none", True, False, False, 0),
    (3, 40, 70, 24, 16, "f32", "gelu", False, True, False, 1),
    (1, 512, 1, 512, 512, "bf16", "none", False, True, False, 0),
    (1, 600, 2, 320, 512, "f32", "silu", True, True, False, 0),
    (2, 777, 1, 1001, 99, "f32", "relu", False, True, False, 0),
    (2, 90, 6, 50, 36, "f32", "gelu", False, True, True, 0),
    (8, 9, 2, 64, 64, "f32", "silu", True, False, True, 0),
    (1, 16, 1, 9000, 72, "bf16", "none", False, False, True, 0),
    (2, 20, 3, 520, 96, "bf16", "silu", True, True, True, 0),
    (1, 64, 1, 1032, 64, "bf16", "relu", True, True, True, 0),
    # large enough for the widest tiles; contraction lengths of whole steps and with a remainder
    (1, 3700, 1, 200, 3640, "bf16", "silu", False, True, True, 0),
    (1, 3700, 1, 384, 1800, "bf16", "gelu", True, True, False, 0),
    (2, 1900, 3, 1100, 1320, "f32", "none", False, False, False, 0),
    (2, 2500, 3, 256, 1856, "bf16", "silu", True, False, True, 0),
    (1, 3700, 1, 140, 3640, "f32", "gelu", False, True, False, 2),
]


@pytest.mark.parametrize("R,rows,G,I,O,dtype,act,gated,bias,residual,off", CASES)
def test_linear_q8(R, rows, G, I, O, dtype, act, gated, bias, residual, off):  # noqa: E741
    import torch
    say(f"linear q8 R={R} rows={rows} G={G} I={I} O={O} {dtype} {act} gated={gated} off={off}")
    N = 2 * O if gated else O
    rng = np.random.default_rng(rows + I)
    (xv, xs), (wv, ws) = _rows8(rng, R, rows, I), _rows8(rng, R, G, N, I)
    ws = (ws * I ** -0.5).astype(np.float32)
    b = round_to(rng.normal(size=(R, G, N)), dtype) if bias else None
    res = round_to(rng.normal(size=(R, rows, O)), dtype) if residual else None
    cnt = _counts(R, G, rows, I) if G > 1 else None
    shape = vr.vrLinearShape(DT[dtype], rows, G, I, O, ACT[act] | (vr.VR_ACT_GATED if gated else 0))
    half = HALF[dtype]
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        x = q8_window(job, (rows, row_bytes(I)), pack(xv, xs), off=4 * off)[0]
        w = q8_window(job, (G, N, row_bytes(I)), pack(wv, ws), off=4 * off)[0]
        out, read = tn.put(shape=(rows, O), fill=5.0)
        gr = None if cnt is None else torch.from_numpy(cnt).cuda()
        vr.vr_linear_q8(job.comm, shape, x, w, out, bias=tn.put(b)[0] if bias else None,
                        residual=tn.put(res)[0] if residual else None, group_rows=gr)
        got = read()
        job.assert_no_async_error()
        for r in range(R):
            c = None if cnt is None else cnt[r]
            xw, ww = xv[r] * xs[r].astype(np.float64)[:, None], wv[r] * ws[r].astype(np.float64)[..., None]
            want, z = L.linear(xw, ww, act, gated, b[r] if bias else None, res[r] if residual else None, c)
            used = L.group_ranges([rows] if c is None else c, rows)[-1][1]
            # the whole-number sum is exact; its conversion, two products and the bias' sum round once each
            product = L.linear(xw, ww, "none", False, None, None, c)[1]
            # the definition itself sums I + 1 products of scaled values in binary64, rounding each and their sum
            mag = L.linear(np.abs(xw), np.abs(ww), "none", False, None, None, c)[1]
            dz = (3 * np.abs(product) + np.abs(z)) * STEP / 2 * 1.01 + mag * (I + 4) * 2.0 ** -53
            a, _ = L.activation(z[:, :O], act)
            da = 1.2 * dz[:, :O] + (np.abs(z[:, :O]) + 1) * ACT_EVAL * (act != "none")  # slopes stay below 1.13
            tol = da * np.abs(z[:, O:]) + (np.abs(a) + da) * dz[:, O:] if gated else da
            tol = tol + np.abs(want) * half + (np.abs(want) + (np.abs(res[r]) if residual else 0)) * 4 * STEP + 2.0 ** -130
            check(got[r, :used], want[:used], tol[:used], "out")
            assert np.all(got[r, used:] == 5.0)  # rows of no group


@pytest.mark.parametrize("rows,I", [(1, 131071), (200, 131071), (300, 128), (40, 1)])
def test_sums_are_exact_at_the_extremes(rows, I):  # noqa: E741
    # every product 2^14: the sum is the largest that fits
    say(f"linear q8: all bytes -128, rows={rows} in={I}")
    O = 20  # noqa: E741
    full = lambda *s: pack(np.full((*s, I), -128, np.int8), np.ones(s, np.float32))  # noqa: E731
    with Job(1) as job:
        x, w = q8_window(job, (rows, row_bytes(I)), full(1, rows))[0], q8_window(job, (O, row_bytes(I)), full(1, O))[0]
        out, read = Tensors(job, "f32").put(shape=(rows, O))
        vr.vr_linear_q8(job.comm, vr.vrLinearShape(0, rows, 1, I, O, 0), x, w, out)
        assert np.all(read() == float(np.float32(16384 * I)))


@pytest.mark.parametrize("rows,O", [(3, 40), (100, 200)])
def test_bytes_behind_the_values_take_no_part(rows, O):  # noqa: E741
    say(f"linear q8: bytes behind the values, rows={rows}")
    I = 101  # noqa: E741
    rng = np.random.default_rng(3)
    (xv, xs), (wv, ws) = _rows8(rng, 1, rows, I), _rows8(rng, 1, 1, O, I)
    outs = []
    for fill in (0, 0x77):
        with Job(1) as job:
            px, pw = pack(xv, xs), pack(wv, ws)
            px[..., I:-4] = fill
            pw[..., I:-4] = fill
            x, w = q8_window(job, px.shape[1:], px)[0], q8_window(job, pw.shape[1:], pw)[0]
            out, read = Tensors(job, "f32").put(shape=(rows, O))
            vr.vr_linear_q8(job.comm, vr.vrLinearShape(0, rows, 1, I, O, 0), x, w, out)
            outs.append(read())
    assert np.array_equal(*outs)


def test_a_poisoned_row_stays_one():
    say("linear q8: scale NaN")
    rows, I, O = 40, 64, 24  # noqa: E741
    rng = np.random.default_rng(3)
    (xv, xs), (wv, ws) = _rows8(rng, 1, rows, I), _rows8(rng, 1, 1, O, I)
    xs[0, 7] = np.nan
    with Job(1) as job:
        for act in ("none", "relu", "gelu", "silu"):
            x, w = q8_window(job, (rows, row_bytes(I)), pack(xv, xs))[0], q8_window(job, (O, row_bytes(I)), pack(wv, ws))[0]
            out, read = Tensors(job, "bf16").put(shape=(rows, O))
            vr.vr_linear_q8(job.comm, vr.vrLinearShape(vr.VR_DT_BF16, rows, 1, I, O, ACT[act]), x, w, out)
            bad = np.isnan(read()[0])
            assert bad[7].all() and not np.delete(bad, 7, 0).any()


@pytest.mark.parametrize("cnt", [[20, -3, 10, 40], [2 ** 31 - 1, 2 ** 31 - 1, 5, 0], [0, 0, 0, -1]])
def test_group_counts_past_the_rows_and_negative(cnt):
    import torch
    say(f"linear q8: bad group counts {cnt}")
    rows, G, I, O = 50, 4, 16, 8  # noqa: E741
    rng = np.random.default_rng(3)
    (xv, xs), (wv, ws) = _rows8(rng, 1, rows, I), _rows8(rng, 1, G, O, I)
    with Job(1) as job:
        x, w = q8_window(job, (rows, row_bytes(I)), pack(xv, xs))[0], q8_window(job, (G, O, row_bytes(I)), pack(wv, ws))[0]
        out, read = Tensors(job, "f32").put(shape=(rows, O), fill=5.0)
        vr.vr_linear_q8(job.comm, vr.vrLinearShape(0, rows, G, I, O, 0), x, w, out,
                        group_rows=torch.tensor([cnt], dtype=torch.int32, device="cuda"))
        assert job.async_error()[1] == vr.VR_ASYNC_CAPACITY
        want, _ = L.linear(xv[0] * xs[0].astype(np.float64)[:, None], wv[0] * ws[0].astype(np.float64)[..., None], "none", False,
                           None, None, cnt)
        used = L.group_ranges(cnt, rows)[-1][1]
        check(read()[0][:used], want[:used], np.abs(want[:used]) * 2 * STEP, "out")
        assert np.all(read()[0][used:] == 5.0)


def test_rows_far_into_a_window():
    # weights past 2^32 bytes: the last group's
    import torch
    say("linear q8: offsets past 32 bits")
    G, I, O, rows = 1024, 4096, 1100, 40  # noqa: E741
    row = row_bytes(I)
    assert (G - 1) * O * row > 1 << 32
    rng = np.random.default_rng(3)
    (xv, xs), (wv, ws) = _rows8(rng, 1, rows, I), _rows8(rng, 2, O, I)
    with Job(1) as job:
        h, views = job.window(G * O * row, fill=0)
        w = views[0].view(G, O, row)
        for i, g in enumerate((0, G - 1)):
            w[g].copy_(torch.from_numpy(pack(wv[i], ws[i])))
        counts = torch.zeros(1, G, dtype=torch.int32)
        counts[0, 0], counts[0, G - 1] = 3, 30
        x = q8_window(job, (rows, row), pack(xv, xs))[0]
        out, read = Tensors(job, "f32").put(shape=(rows, O), fill=5.0)
        vr.vr_linear_q8(job.comm, vr.vrLinearShape(0, rows, G, I, O, 0), x, (h, 0), out, group_rows=counts.cuda())
        got = read()[0]
        for i, (a, b) in enumerate(((0, 3), (3, 33))):
            want = (xv[0, a:b].astype(np.float64) @ wv[i].astype(np.float64).T) * xs[0, a:b, None] * ws[i][None]
            check(got[a:b], want, np.abs(want) * 2 * STEP, "out")
        assert np.all(got[33:] == 5.0)
        job.assert_no_async_error()


def test_residual_in_place_no_rows_and_refusals():
    import torch
    say("linear q8: residual in place, no rows, refusals")
    R, rows, I, O = 2, 40, 130, 24  # noqa: E741
    rng = np.random.default_rng(3)
    (xv, xs), (wv, ws) = _rows8(rng, R, rows, I), _rows8(rng, R, 1, O, I)
    res = round_to(rng.normal(size=(R, rows, O)), "f32")
    S = vr.vrLinearShape
    ok = S(vr.VR_DT_F32, rows, 1, I, O, vr.VR_ACT_SILU)
    with Job(R) as job:
        tn = Tensors(job, "f32")
        x, w = q8_window(job, (rows, row_bytes(I)), pack(xv, xs))[0], q8_window(job, (O, row_bytes(I)), pack(wv, ws))[0]
        out, read = tn.put(shape=(rows, O))
        place, place_read = tn.put(res)
        vr.vr_linear_q8(job.comm, ok, x, w, out, residual=tn.put(res)[0])
        vr.vr_linear_q8(job.comm, ok, x, w, place, residual=place)
        assert np.array_equal(read(), place_read())
        call = lambda s, *a, **k: (lambda: vr.vr_linear_q8(job.comm, s, *a, **k))  # noqa: E731
        for bad in (S(2, rows, 1, I, O, 0), S(0, -1, 1, I, O, 0), S(0, rows, 0, I, O, 0), S(0, rows, 1025, I, O, 0),
                    S(0, rows, 1, 0, O, 0), S(0, rows, 1, I, 0, 0), S(0, rows, 1, I, O, 4), S(0, rows, 2, I, O, 0),
                    S(0, rows + 64, 1, I, O, 0), S(0, rows, 1, 131072, O, 0), S(0, rows, 1, I, O + 9, 0)):
            refused(call(bad, x, w, out))
        refused(call(ok, None, w, out))
        refused(call(ok, x, None, out))
        refused(call(ok, x, w, None))
        refused(call(ok, x, w, (x.window, 0)))
        refused(call(ok, x, w, out, residual=(out.window, out.offset + 4)))
        refused(call(ok, (x.window, x.offset + 2), w, out))
        refused(call(ok, x, (w.window, w.offset + 1), out))
        refused(call(ok, x, w, (out.window, out.offset + 2)))
        refused(call(ok, x, w, out, group_rows=torch.zeros(R, 1, dtype=torch.int32)))  # host memory
        sw, _ = job.window(1 << 14, flags=vr.VR_WIN_STRICT_ORDERING)
        vr.vr_va_signal_reset(job.comm, sw, 0, 64)
        refused(call(ok, x, w, (sw, 0)), vr.VR_ERR_INVALID_USAGE)
        call(S(0, 0, 1, I, O, 0), x, w, out)()
        job.assert_no_async_error()
