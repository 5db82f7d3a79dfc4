"""Pins of the norm, rows in 8 bits and the combine's gradient in oracle/layers.py: hand-worked cases, torch's autograd
on the CPU and central differences; and the binding's host-only calls."""
import numpy as np
import pytest
import torch

import collective_window_put_amd as vr
from oracle import layers as L


def test_norm_by_hand():
    assert np.allclose(L.norm([[3.0, 4.0]], [2.0, 1.0], 0.0), [[3 * 2 / 12.5 ** 0.5, 4 / 12.5 ** 0.5]])
    assert np.allclose(L.norm([[0.0, 0.0]], None, 1e-5), 0.0)
    assert np.allclose(L.norm([[1.0]], None, 3.0), 0.5)


@pytest.mark.parametrize("gain,more", [(True, True), (False, False)])
def test_norm_gradient_against_autograd_and_differences(gain, more):
    rng = np.random.default_rng(1)
    h, g, d, s = rng.normal(size=(5, 7)), rng.normal(size=7), rng.normal(size=(5, 7)), rng.normal(size=(5, 7))
    th, tg = torch.tensor(h, requires_grad=True), torch.tensor(g, requires_grad=True)
    y = th * torch.rsqrt((th * th).mean(-1, keepdim=True) + 0.01) * (tg if gain else torch.ones(7) * tg / tg.detach())
    assert np.allclose(y.detach().numpy(), L.norm(h, g if gain else None, 0.01), atol=1e-14)
    (y * torch.tensor(d)).sum().backward()
    dh, dg = L.norm_backward(d, h, g if gain else None, 0.01, s if more else None)
    assert np.allclose(dh - (s if more else 0), th.grad.numpy(), atol=1e-13)
    assert np.allclose(dg, tg.grad.numpy() * (1 if gain else g), atol=1e-13)
    e = 1e-6
    for at in np.ndindex(*h.shape):
        up, down = h.copy(), h.copy()
        up[at] += e
        down[at] -= e
        f = lambda v: float((L.norm(v, g if gain else None, 0.01) * d).sum())  # noqa: E731
        assert abs((f(up) - f(down)) / (2 * e) - (dh[at] - (s[at] if more else 0))) < 1e-8


def test_rows_in_8_bits_by_hand():
    v, s = L.to_8_bits([[127.0, -127.0, 0.5, 1.5, -2.5, 63.2], [0, 0, 0, 0, 0, 0], [1e-37, 0, 0, 0, 0, -1e-37],
                        [np.nan, 1, 2, 3, 4, 5], [1, 2, -np.inf, 3, 4, 5]])
    assert v.tolist() == [[127, -127, 0, 2, -2, 63], [0] * 6, [0] * 6, [0] * 6, [0] * 6]  # halves to the even
    assert s[0] == 1 and s[1] == 0 and s[2] == 0 and np.isnan(s[3]) and np.isnan(s[4])


def test_rows_in_8_bits_are_within_half_a_scale():
    x = (np.random.default_rng(2).normal(size=(50, 33)) * 10.0 ** np.arange(-25, 25)[:, None]).astype(np.float32)
    v, s = L.to_8_bits(x)
    off = np.abs(v.astype(np.float64) * s[:, None] - x)
    # half a step, and the roundings of scale, of the multiplier and of the step itself
    assert np.all(off <= s[:, None] * (0.5 + 128 * 3 * 2.0 ** -24)) and np.all(np.abs(v).max(-1) == 127)


def test_combine_gradient_against_autograd():
    rng = np.random.default_rng(3)
    S, T, K, H = 2, 3, 2, 4
    rank, row = rng.integers(0, 2, (S, T, K)), np.arange(S * T * K).reshape(S, T, K)
    rank[0, 1, 0] = row[0, 1, 0] = -1
    y, w, d = rng.normal(size=(2, S * T * K, H)), rng.normal(size=(S, T, K)), rng.normal(size=(S, T, H))
    ty, tw = torch.tensor(y, requires_grad=True), torch.tensor(w, requires_grad=True)
    out = torch.zeros(S, T, H, dtype=torch.float64)
    for s, t, k in np.ndindex(S, T, K):
        if row[s, t, k] >= 0:
            out[s, t] = out[s, t] + tw[s, t, k] * ty[rank[s, t, k], row[s, t, k]]
    (out * torch.tensor(d)).sum().backward()
    dy, dw = L.combine_backward(d, y, rank, row, w)
    assert len(dy) == S * T * K - 1 and np.allclose(dw, tw.grad.numpy(), atol=1e-14)
    whole = np.zeros_like(y)
    for at, v in dy.items():
        whole[at] = v
    assert np.allclose(whole, ty.grad.numpy(), atol=1e-14)


def test_sizes_that_the_host_computes():
    assert [vr.vr_q8_row_bytes(c) for c in (1, 124, 125, 128, 252, 253, 512, 4096)] == [128, 128, 256, 256, 256, 384, 640, 4224]
    assert vr.vr_q8_row_bytes(0) == vr.vr_q8_row_bytes(-5) == vr.vr_q8_row_bytes((1 << 20) + 1) == 0
    N = vr.vrNormShape
    assert vr.vr_norm_backward_workspace_bytes(2, N(0, 100, 64, 1e-5)) > 0
    for bad in (N(2, 100, 64, 1e-5), N(0, -1, 64, 1e-5), N(0, 1 + (1 << 24), 64, 1e-5), N(0, 100, 0, 1e-5),
                N(0, 100, 1 + (1 << 20), 1e-5), N(0, 100, 64, 0.0), N(0, 100, 64, -1.0), N(0, 100, 64, float("nan")),
                N(0, 100, 64, float("inf")), N(0, 100, 64, 1e-39)):
        assert vr.vr_norm_backward_workspace_bytes(2, bad) == 0
    assert vr.vr_norm_backward_workspace_bytes(0, N(0, 100, 64, 1e-5)) == 0


def test_calls_without_a_communicator_are_refused():
    x = (1, 0)
    for call in (lambda: vr.vr_norm(0, vr.vrNormShape(0, 1, 1, 1e-5), x, out=x, stream=0),
                 lambda: vr.vr_norm_backward(0, vr.vrNormShape(0, 1, 1, 1e-5), x, x, dh=x, stream=0),
                 lambda: vr.vr_quantize(0, x, 0, 1, 1, x, stream=0), lambda: vr.vr_dequantize(0, x, 0, 1, 1, x, stream=0),
                 lambda: vr.vr_linear_q8(0, vr.vrLinearShape(0, 1, 1, 1, 1, 0), x, x, x, stream=0),
                 lambda: vr.vr_combine_backward(0, x, x, 1, 4, 0, 1, 1, 1, 1, 1, 1, dy=x, stream=0)):
        with pytest.raises(vr.VrError) as e:
            call()
        assert e.value.code == vr.VR_ERR_INVALID_ARGUMENT
