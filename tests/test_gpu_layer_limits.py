"""Shapes of many tiles and little memory: more workgroups than one launch may
have threads for (2^32 in a direction)."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say

pytestmark = pytest.mark.gpu


def _window(job, shape):
    """(tensors of every rank, slice), zeros, bf16."""
    import torch
    n = torch.Size(shape).numel()
    h, views = job.window(n * 2, fill=0)
    return [v.view(torch.bfloat16).view(shape) for v in views], vr.vrSlice(h, 0)


def _normal(t, seed):
    import torch
    t.copy_(torch.randn(t.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))


def test_few_rows_of_many_groups_and_columns():
    # 16 rows, 1024 groups, 131088 columns: 1025 * 8193 workgroups of 512 threads, past 2^32
    import torch
    rows, G, I, O = 16, 1024, 1, 131088
    assert (rows // 16 + G) * (O // 16) * 512 > 1 << 32
    say("linear: few rows, 1024 groups of 131088 columns")
    counts = torch.zeros(1, G, dtype=torch.int32)
    held = [(0, 3), (511, 5), (1022, 1), (1023, 6)]
    for g, n in held:
        counts[0, g] = n
    with Job(1) as job:
        x, xs = _window(job, (rows, I))
        w, ws = _window(job, (G, O, I))
        out, outs = _window(job, (rows, O))
        _normal(x[0], 1)
        for g, _ in held:
            _normal(w[0][g], g + 2)
        out[0].fill_(5.0)
        shape = vr.vrLinearShape(vr.VR_DT_BF16, rows, G, I, O, vr.VR_ACT_NONE)
        vr.vr_linear(job.comm, shape, xs, ws, outs, group_rows=counts.cuda())
        torch.cuda.synchronize()
        at = 0
        for g, n in held:  # one product each, exact in binary32
            want = (x[0][at:at + n].float() * w[0][g].float().view(1, O)).bfloat16()
            assert torch.equal(out[0][at:at + n], want), g
            at += n
        assert bool((out[0][at:] == 5.0).all())
        job.assert_no_async_error()


def test_gradients_of_many_groups_and_inputs():
    # 4 ranks, 1024 groups, 2^20 inputs, one output: 2^25 tiles of 128 x 128, 256 threads each
    import torch
    R, rows, G, I, O = 4, 2, 1024, 1 << 20, 1
    assert R * G * (I // 128) * 256 > 1 << 32
    say("linear gradients: 4 ranks, 1024 groups of 2^20 inputs")
    counts = torch.zeros(R, G, dtype=torch.int32)
    held = {r: ((0, 3 * r), (1, G - 1 - r)) for r in range(R)}  # row, group
    for r, pairs in held.items():
        for _, g in pairs:
            counts[r, g] += 1
    with Job(R) as job:
        x, xs = _window(job, (rows, I))
        w, ws = _window(job, (G, O, I))
        dout, ds = _window(job, (rows, O))
        dx, dxs = _window(job, (rows, I))
        dw, dws = _window(job, (G, O, I))
        for r in range(R):
            _normal(x[r], r)
            _normal(dout[r], 10 + r)
            dx[r].fill_(5.0)
            dw[r].fill_(5.0)
            for row, g in held[r]:
                _normal(w[r][g], 20 + 2 * r + row)
        shape = vr.vrLinearShape(vr.VR_DT_BF16, rows, G, I, O, vr.VR_ACT_NONE)
        need = vr.vr_linear_backward_workspace_bytes(R, shape)
        room = torch.empty(need, dtype=torch.uint8, device="cuda")
        vr.vr_linear_backward(job.comm, shape, ds, xs, ws, dx=dxs, dw=dws, group_rows=counts.cuda(), workspace=room,
                              workspace_bytes=need)
        torch.cuda.synchronize()
        for r in range(R):
            for row, g in held[r]:
                d = dout[r][row].float()
                assert torch.equal(dx[r][row], (d * w[r][g][0].float()).bfloat16()), (r, row)
                assert torch.equal(dw[r][g][0], (d * x[r][row].float()).bfloat16()), (r, g)
                dw[r][g].zero_()
            assert not bool(dw[r].any()), r  # groups without rows
        job.assert_no_async_error()


def _moe(job, T, E, K, H, I):
    """Tensors of a few-token layer of relu experts, one rank, and a function that runs it."""
    import torch
    t = {k: _window(job, s) for k, s in dict(x=(T, H), up=(E, I, H), down=(E, H, I), out=(T, H)).items()}
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(1, T, K, dtype=torch.int32, device="cuda")
    weights = torch.zeros(1, T, K, device="cuda")
    shape = vr.vrMoeShape(vr.VR_DT_BF16, T, H, I, E, K, vr.VR_ACT_RELU, vr.VR_ROUTE_RENORM)
    need = vr.vr_moe_layer_workspace_bytes(1, shape)
    room = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run():
        vr.vr_moe_layer(job.comm, shape, t["x"][1], router, t["up"][1], t["down"][1], t["out"][1], idx, weights,
                        workspace=room, workspace_bytes=need)
        torch.cuda.synchronize()
        job.assert_no_async_error()
    return {k: v[0][0] for k, v in t.items()}, router, idx[0], weights[0], run


def test_few_token_layer_of_many_experts_and_inner_columns():
    # 1024 experts of 131104 inner columns: 8194 * 1024 workgroups of 512 threads for the up product
    import torch
    T, E, K, H, I = 64, 1024, 16, 6, 131104  # noqa: E741
    assert E * (I // 16) * 512 > 1 << 32
    say("moe layer: 1024 experts of 131104 inner columns")
    with Job(1) as job:
        t, router, idx, weights, run = _moe(job, T, E, K, H, I)
        # token n is the signs of n's bits; experts n K .. n K + K - 1 look like it (logit 6, others 4 or less)
        signs = (torch.arange(T, device="cuda")[:, None] >> torch.arange(H, device="cuda") & 1) * 2.0 - 1.0
        t["x"].copy_(signs)
        router.copy_(signs.repeat_interleave(K, 0))
        for name, seed in (("up", 2), ("down", 3)):  # every column adds something positive to its token's sum
            _normal(t[name], seed)
            t[name].abs_()
        t["up"].mul_(router[:, None, :])
        t["down"].mul_(I ** -1)
        run()
        for n in range(T):
            e = idx[n].long()
            assert e.tolist() == list(range(n * K, (n + 1) * K))
            h = (t["up"][e].double() * t["x"][n].double()).sum(-1)
            want = (weights[n].double()[:, None] * (t["down"][e].double() * h[:, None]).sum(-1)).sum(0)
            # sums of H, 2 I and K positive products, a step each; h held to 2^-16; one rounding to bf16
            tol = want * ((2 * I + 2 * K + H + 8) * 2.0 ** -23 + 2.0 ** -16 + 2.0 ** -8)
            assert bool(((t["out"][n].double() - want).abs() <= tol).all()), n


def test_few_token_layer_of_many_experts_and_hidden_elements():
    # 1024 experts of 2^20 hidden elements: 8192 * 1024 workgroups of 512 threads for the down product
    import torch
    T, E, K, H, I = 16, 1024, 64, 1 << 20, 1  # noqa: E741
    assert E * (H // 128) * 512 >= 1 << 32
    say("moe layer: 1024 experts of 2^20 hidden elements")
    with Job(1) as job:
        t, router, idx, weights, run = _moe(job, T, E, K, H, I)
        # token n is the unit vector of element n, which alone counts in its logits and its inner value
        for n in range(T):
            t["x"][n, n] = 1.0
            router[n * K:(n + 1) * K, n] = 1.0
        gen = torch.Generator(device="cuda").manual_seed(4)
        t["up"][:, 0, :T] = 1.0 + torch.rand((E, T), generator=gen, device="cuda").bfloat16()
        for e in range(E):
            t["down"][e, :, 0].normal_(generator=gen)
        run()
        for n in range(T):
            e = idx[n].long()
            assert sorted(e.tolist()) == list(range(n * K, (n + 1) * K))
            terms = weights[n].double()[:, None] * t["down"][e, :, 0].double() * t["up"][e, 0, n].double()[:, None]
            want = terms.sum(0)
            # K products and sums, a step each, and one rounding to bf16
            tol = terms.abs().sum(0) * (K + 8) * 2.0 ** -23 + want.abs() * 2.0 ** -8
            assert bool(((t["out"][n].double() - want).abs() <= tol).all()), n
