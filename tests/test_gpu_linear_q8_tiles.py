"""The product of rows in 8 bits where a workgroup takes 256 x 256 tile after tile (k_gemm_run): every type and epilogue,
ragged rows, columns and contraction, no whole step to many, one group and many on several ranks. Sizes follow from the rule
that chooses the tile, which is asserted, and are of more tiles than workgroups, so that a tile's loads run ahead of the
one before. (Of the sizes in test_gpu_linear_q8.py two dense ones take such tiles, fewer than there are workgroups; its
others take smaller ones.)"""
import math

import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import ACT, ACT_EVAL, DT, HALF, STEP
from rows_util import row_bytes

pytestmark = pytest.mark.gpu
WORKGROUPS = 256


def tiles(n, R, rows, G, O, gated, counts):  # noqa: E741
    """n x n tiles to expect, as the library counts them: a group's last row tile is half empty."""
    cols = -(-O // (n // 2 if gated else n))
    return R * (rows // n + (G + 1) // 2 if counts else -(-rows // n)) * cols


def takes_tile_after_tile(*shape):
    wide, small = tiles(256, *shape), tiles(128, *shape)
    return -(-wide // 256) * 100 <= -(-small // 512) * 59


CASES = [  # R, rows, G, I, O, dtype, act, gated, bias, residual
    # dense, bias and residual behind the counted wait; 1, 0, 1 and a bit, 2, many steps; a ragged last row and column of tiles
    (1, 7900, 1, 256, 4090, "bf16", "gelu", False, True, True),
    (1, 7900, 1, 100, 4090, "bf16", "relu", False, True, True),
    (1, 7900, 1, 128, 4090, "bf16", "silu", False, True, False),
    (1, 7900, 1, 200, 4090, "bf16", "none", False, False, True),
    (1, 7900, 1, 1064, 4090, "bf16", "none", False, False, False),
    (1, 7900, 1, 256, 4090, "f32", "gelu", False, True, True),
    (1, 7900, 1, 60, 4090, "f32", "none", False, True, True),
    (1, 7900, 1, 128, 4090, "f32", "relu", False, False, True),
    (1, 7900, 1, 328, 4090, "f32", "silu", False, False, False),
    (1, 7936, 1, 640, 4096, "f32", "none", False, False, False),  # whole tiles alone
    (1, 7936, 1, 640, 4096, "bf16", "silu", False, True, True),
    # gated
    (1, 7900, 1, 256, 2045, "bf16", "silu", True, True, True),
    (1, 7900, 1, 136, 2045, "bf16", "none", True, True, False),
    (1, 7900, 1, 300, 2045, "f32", "gelu", True, True, True),
    (1, 7900, 1, 512, 2045, "f32", "relu", True, False, False),
    # by expert on several ranks: ragged groups, some empty, rows of no group behind the last
    (3, 8000, 5, 256, 520, "bf16", "silu", True, True, True),
    (3, 8000, 5, 392, 520, "f32", "silu", True, True, True),
    (4, 10000, 5, 100, 520, "bf16", "gelu", False, True, True),
    (4, 10000, 5, 264, 520, "f32", "none", False, True, True),
    (8, 10000, 32, 140, 500, "bf16", "relu", True, False, True),
    (3, 13000, 66, 200, 440, "bf16", "none", False, True, True),  # a table of more groups than lanes
]


def _act(z, name):
    import torch
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z.clamp(min=0) if name == "relu" else z


@pytest.mark.parametrize("R,rows,G,I,O,dtype,act,gated,bias,residual", CASES)
def test_tile_after_tile(R, rows, G, I, O, dtype, act, gated, bias, residual):  # noqa: E741
    import torch
    say(f"linear q8, tile after tile: R={R} rows={rows} G={G} I={I} O={O} {dtype} {act} gated={gated} {bias} {residual}")
    shape = (R, rows, G, O, gated, G > 1)
    assert takes_tile_after_tile(*shape) and tiles(256, *shape) > WORKGROUPS
    N, tt, half = 2 * O if gated else O, torch.float32 if dtype == "f32" else torch.bfloat16, HALF[dtype]
    gen = torch.Generator(device="cuda").manual_seed(rows + I)
    with Job(R) as job:
        def q8(*lead):
            n, rb = math.prod(lead), row_bytes(I)
            h, views = job.window(n * rb, fill=0)
            for v in views:
                t = v.view(n, rb)
                t[:, :I] = torch.randint(-127, 128, (n, I), generator=gen, device="cuda", dtype=torch.int8).view(torch.uint8)
                s = (torch.rand(n, 1, generator=gen, device="cuda") + 0.5) / 74 * I ** -0.25
                t[:, -4:] = s.view(torch.uint8)
            return vr.vrSlice(h, 0), [v.view(*lead, rb) for v in views]

        def plain(*dims, fill=None):
            n = math.prod(dims)
            h, views = job.window(n * tt.itemsize, fill=None)
            got = [v.view(tt).view(dims) for v in views]
            for t in got:
                t.copy_(torch.randn(dims, generator=gen, device="cuda")) if fill is None else t.fill_(fill)
            return vr.vrSlice(h, 0), got

        (x, xt), (w, wt) = q8(rows), q8(G, N)
        b, bt = plain(G, N) if bias else (None, None)
        res, rt = plain(rows, O) if residual else (None, None)
        out, ot = plain(rows, O, fill=5.0)
        counts = None
        if G > 1:
            rng = np.random.default_rng(rows)
            share = rng.uniform(0.1, 1, size=(R, G)) * (rng.random((R, G)) > 0.15)
            share[:, 0] += 0.1
            counts = np.floor(share / share.sum(1, keepdims=True) * (rows - 77)).astype(np.int32)
        gr = None if counts is None else torch.from_numpy(counts).cuda()
        call = lambda: vr.vr_linear_q8(job.comm, vr.vrLinearShape(DT[dtype], rows, G, I, O, ACT[act] | (vr.VR_ACT_GATED if gated else 0)),  # noqa: E731
                                       x, w, out, bias=b, residual=res, group_rows=gr)
        call()
        torch.cuda.synchronize()
        scale = lambda t: t[..., -4:].contiguous().view(torch.float32).double()  # noqa: E731
        for r in range(R):
            at = 0
            for g, n in enumerate([rows] if counts is None else counts[r].tolist()):
                rx, rw = xt[r][at:at + n], wt[r][g]
                # whole numbers below 2^53: exact, whatever the order
                p = rx[:, :I].view(torch.int8).double() @ rw[:, :I].view(torch.int8).double().T.contiguous()
                p = p * scale(rx) * scale(rw).T
                z = p + bt[r][g].double() if bias else p
                # the sum's conversion, two products and the bias' sum round once each; the activation, whose slope is below 1.13
                dz = (3 * p.abs() + z.abs()) * STEP / 2 * 1.01
                a = _act(z[:, :O], act)
                da = 1.2 * dz[:, :O] + (z[:, :O].abs() + 1) * ACT_EVAL * (act != "none")
                if dtype == "bf16" and act in ("gelu", "silu"):
                    da = da + a.abs() * 2.0 ** -11  # bf16's arithmetic: 2^-12 of the value for the tail, and exp2 and rcp's steps
                want, tol = (a * z[:, O:], da * z[:, O:].abs() + (a.abs() + da) * dz[:, O:]) if gated else (a, da)
                more = rt[r][at:at + n].double() if residual else torch.zeros((), dtype=torch.float64, device="cuda")
                want = want + more
                tol = tol + want.abs() * half + (want.abs() + more.abs()) * 4 * STEP + 2.0 ** -130
                bad = ~((ot[r][at:at + n].double() - want).abs() <= tol)
                assert not bool(bad.any()), (r, g, int(bad.sum()), bad.nonzero()[:3].tolist())
                at += n
            assert bool((ot[r][at:] == 5).all())  # rows of no group
        first = [t.clone() for t in ot]
        for rep in range(4):  # and every time the same
            for t in ot:
                t.fill_(5)
            call()
            assert all(torch.equal(t, f) for t, f in zip(ot, first)), rep
        job.assert_no_async_error()
