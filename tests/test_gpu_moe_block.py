"""The example's block: its training step against autograd in binary64, and its serving step in 8 bits stage by stage,
each from what the stage before left."""
import os
import sys

import numpy as np
import pytest

from gpu_util import say
from layer_util import ACT_EVAL, STEP
from oracle import layers as L
from rows_util import pack, unpack

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _block(R, T, H, I, E, K, seed):  # noqa: E741
    import torch

    from moe_step import MoeBlock
    gen = torch.Generator().manual_seed(seed)
    b = MoeBlock(R, T, H, I, E, K, torch.float32)
    n = lambda t, s=1.0: t.copy_(torch.randn(t.shape, generator=gen) * s)  # noqa: E731
    n(b.branch), n(b.residual), n(b.dout), n(b.dstream), n(b.w_up, H ** -0.5), n(b.w_down, I ** -0.5)
    n(b.gain, 0.3)
    b.gain += 1
    n(b.router, 2 * H ** -0.5)
    b.router.copy_(b.router[:1].expand_as(b.router).clone())  # one router, on every rank
    return b


@pytest.mark.parametrize("R,T,H,I,E,K", [(1, 24, 40, 24, 4, 2), (4, 7, 36, 20, 8, 3)])
def test_training_step_against_autograd(R, T, H, I, E, K):  # noqa: E741
    import torch
    say(f"moe block R={R} T={T} H={H} I={I} E={E} K={K}")
    b = _block(R, T, H, I, E, K, R * T)
    b.forward()
    b.backward()
    b.check()
    branch, residual, gain, router, up, down = (t.detach().cpu().double().requires_grad_() for t in (
        b.branch, b.residual, b.gain, b.router, b.w_up, b.w_down))
    stream = branch + residual
    x = stream * torch.rsqrt((stream * stream).mean(-1, keepdim=True) + b.EPS) * gain[:, None]
    p = torch.softmax(torch.einsum("rth,reh->rte", x, router[:, 0]), -1)
    top = b.topk.cpu().long()  # the device's choice: a tie within rounding may go either way
    p = p.gather(-1, top)
    p = p / p.sum(-1, keepdim=True)
    u, d = up.reshape(E, 2 * I, H)[top], down.reshape(E, H, I)[top]
    z = torch.einsum("rtkuh,rth->rtku", u, x)
    out = (p[..., None] * torch.einsum("rtkhi,rtki->rtkh", d, torch.nn.functional.silu(z[..., :I]) * z[..., I:])).sum(2)
    (out * b.dout.cpu().double()).sum().add((stream * b.dstream.cpu().double()).sum()).backward()
    # every value is a chain of sums of at most H, I, E, rows or 2 I terms and a few operations on each; a sum is off by its
    # length in steps of its terms' size, which no entry's own size bounds: the largest one's does, sixteen times
    tol = 16 * (3 * H + 3 * I + E + R * T * K + 128) * STEP
    for name, got, want in (("stream", b.stream, stream), ("out", b.out, out), ("dbranch", b.dbranch, branch.grad),
                            ("dgain", b.dgain, gain.grad), ("drouter", b.drouter, router.grad), ("dw_up", b.dw_up, up.grad),
                            ("dw_down", b.dw_down, down.grad)):
        off = (got.cpu().double() - want.detach()).abs().max()
        assert float(off) <= tol * float(want.detach().abs().max()), (name, float(off), tol)
    assert torch.equal(branch.grad, residual.grad)
    b.close()


def _wide(rows, cols):
    v, s = unpack(rows, cols)
    return v.astype(np.float64) * s.astype(np.float64)[..., None]


@pytest.mark.parametrize("R,T,H,I,E,K", [(1, 24, 40, 24, 4, 2), (4, 17, 260, 132, 8, 3)])
def test_serving_step_in_8_bits(R, T, H, I, E, K):  # noqa: E741
    import torch
    say(f"moe block in 8 bits R={R} T={T} H={H} I={I} E={E} K={K}")
    b = _block(R, T, H, I, E, K, R * T + 1)
    b.quantize_weights()
    b.serve()
    b.check()
    G = E // R
    f = lambda t: t.cpu().numpy()  # noqa: E731
    up, down = f(b.w_up8).reshape(R, G, 2 * I, -1), f(b.w_down8).reshape(R, G, H, -1)
    for r in range(R):
        assert np.array_equal(f(b.w_up8)[r], pack(*L.to_8_bits(f(b.w_up)[r].reshape(-1, H))))
        assert np.array_equal(f(b.w_down8)[r], pack(*L.to_8_bits(f(b.w_down)[r].reshape(-1, I))))
    x8, recv8, topk, pos, counts = f(b.x8), f(b.recv8), f(b.topk), f(b.pos), f(b.counts)
    x, s = _wide(x8, H), unpack(x8, H)[1].astype(np.float64)[..., None]
    assert np.all(np.abs(x - f(b.x)) <= s * (0.5 + 127 * 4 * STEP))  # the same norm, in 8 bits and whole
    for at in np.ndindex(R, T, K):  # one dispatch took values and scales along
        assert np.array_equal(recv8[topk[at] // G, pos[at]], x8[at[:2]])
    h, y, out = f(b.h).astype(np.float64), f(b.y).astype(np.float64), f(b.out).astype(np.float64)
    for r in range(R):
        used = int(counts[r].sum())
        want, z = L.linear(_wide(recv8[r], H), _wide(up[r], H), "silu", True, None, None, counts[r])
        mag = L.linear(np.abs(_wide(recv8[r], H)), np.abs(_wide(up[r], H)), "none", False, None, None, counts[r])[1]
        dz = np.abs(z) * 4 * STEP + mag * (H + 4) * 2.0 ** -53
        da = 1.2 * dz[:, :I] + (np.abs(z[:, :I]) + 1) * ACT_EVAL
        tol = da * np.abs(z[:, I:]) + (np.abs(L.activation(z[:, :I], "silu")[0]) + da) * dz[:, I:] + np.abs(want) * 2 * STEP
        assert np.all(np.abs(h[r] - want)[:used] <= tol[:used] + 2.0 ** -130)
        h8 = f(b.h8)[r]
        assert np.array_equal(h8[:used], pack(*L.to_8_bits(f(b.h)[r, :used])))
        want, _ = L.linear(_wide(h8, I), _wide(down[r], I), "none", False, None, None, counts[r])
        mag = L.linear(np.abs(_wide(h8, I)), np.abs(_wide(down[r], I)), "none", False, None, None, counts[r])[0]
        assert np.all(np.abs(y[r] - want)[:used] <= (np.abs(want) * 4 * STEP + mag * (I + 4) * 2.0 ** -53)[:used] + 2.0 ** -130)
    w = f(b.weights).astype(np.float64)
    terms = w[..., None] * y[topk // G, pos]
    assert np.all(np.abs(out - terms.sum(2)) <= np.abs(terms).sum(2) * (K + 2) * STEP)
    # and the whole is the unquantized layer's, but for what 8 bits lose: each of three rounded operands is off by half a
    # scale, 1 / 254 of its row's largest value, about 3.5 of its size: uniform errors of 0.4 %, 1.1 % for the product of two
    # and 1.5 % along the chain; twice that is a wrong formula
    b.forward()
    assert torch.equal(b.topk.cpu(), torch.from_numpy(topk))
    whole = f(b.out).astype(np.float64)
    assert np.linalg.norm(out - whole) <= 0.03 * np.linalg.norm(whole)
    b.close()


def test_the_example_runs(capsys):
    import moe_step
    say("examples/moe_step.py")
    moe_step.main()
    assert "block in 8 bits" in capsys.readouterr().out
