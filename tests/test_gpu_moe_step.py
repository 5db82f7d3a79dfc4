"""The example's training step and decoding step against autograd in binary64."""
import os
import sys

import pytest

from gpu_util import say
from layer_util import STEP
from oracle import layers as L

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("R,T,H,I,E,K", [(1, 24, 40, 24, 4, 2), (4, 7, 36, 20, 8, 3)])
def test_step_against_autograd(R, T, H, I, E, K):  # noqa: E741
    import torch

    from moe_step import MoeStep
    say(f"moe step R={R} T={T} H={H} I={I} E={E} K={K}")
    gen = torch.Generator().manual_seed(R * T)
    step = MoeStep(R, T, H, I, E, K, torch.float32)
    n = lambda t, s=1.0: t.copy_(torch.randn(t.shape, generator=gen) * s)  # noqa: E731
    n(step.x), n(step.dout), n(step.logits), n(step.w_up, H ** -0.5), n(step.w_down, I ** -0.5)
    step.forward()
    step.backward()
    step.check()
    x, logits, up, down = (t.detach().cpu().double().requires_grad_() for t in (step.x, step.logits, step.w_up, step.w_down))
    top = torch.from_numpy(L.route(logits.detach().numpy(), K, True)[0]).long()
    assert torch.equal(step.topk.cpu().long(), top)
    p = torch.softmax(logits, -1).gather(-1, top)
    p = p / p.sum(-1, keepdim=True)
    u, d = up.reshape(E, 2 * I, H)[top], down.reshape(E, H, I)[top]  # [R, T, K, ...]
    z = torch.einsum("rtkuh,rth->rtku", u, x)
    h = torch.nn.functional.silu(z[..., :I]) * z[..., I:]
    out = (p[..., None] * torch.einsum("rtkhi,rtki->rtkh", d, h)).sum(2)
    out.backward(step.dout.cpu().double())
    # every value is a chain of sums of at most H, I, rows or 2 I terms and the weights' few operations; each sum is off
    # by its length in steps of its terms' size, which no entry's own size bounds: the largest one's does, eight times
    tol = 8 * (H + 3 * I + R * T * K + 64) * STEP
    for name, got, want in (("out", step.out, out), ("dx", step.dx, x.grad), ("dw_up", step.dw_up, up.grad),
                            ("dw_down", step.dw_down, down.grad), ("dlogits", step.dlogits, logits.grad)):
        off = (got.cpu().double() - want.detach()).abs().max()
        assert float(off) <= tol * float(want.detach().abs().max()), name
    step.close()


def test_decoding_takes_the_same_path():
    import torch

    from moe_step import MoeStep
    say("moe step: a few tokens in one call")
    R, T, H, I, E, K = 2, 6, 64, 32, 8, 2  # noqa: E741
    gen = torch.Generator().manual_seed(3)
    step = MoeStep(R, T, H, I, E, K, torch.float32)
    n = lambda t, s=1.0: t.copy_(torch.randn(t.shape, generator=gen) * s)  # noqa: E731
    n(step.x), n(step.w_up, H ** -0.5), n(step.w_down, I ** -0.5)
    router = (torch.randn(E, H, generator=gen) * H ** -0.5).cuda()
    step.logits.copy_((step.x.double() @ router.double().t()).float())
    step.forward()
    out, idx, weights = step.decode(T, router)
    step.check()
    assert torch.equal(idx, step.topk)
    tol = 8 * (H + 2 * I + 64) * STEP
    assert float((weights - step.weights).abs().max()) <= tol
    assert float((out - step.out).abs().max()) <= 2 * tol * float(step.out.abs().max())
    step.close()
