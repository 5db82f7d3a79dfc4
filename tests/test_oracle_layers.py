"""Pins of oracle/layers.py: hand-worked cases, torch's functions on the CPU,
and central differences for the gradients."""
import numpy as np
import pytest
import torch

from oracle import layers as L


def test_route_by_hand():
    idx, w = L.route(np.array([[0.0, np.log(3.0), 0.0, -np.inf]]), 3, False)
    assert idx.tolist() == [[1, 0, 2]]  # the tie goes to the lowest index
    assert np.allclose(w, [[0.6, 0.2, 0.2]], atol=1e-15)
    idx, w = L.route(np.array([[0.0, np.log(3.0), 0.0, -np.inf]]), 2, True)
    assert idx.tolist() == [[1, 0]] and np.allclose(w, [[0.75, 0.25]], atol=1e-15)


def test_route_masks_leave_nothing():
    idx, w = L.route(np.array([[-np.inf, np.nan, np.inf], [-np.inf, 2.0, -np.inf]]), 2, True)
    assert idx.tolist() == [[-1, -1], [1, -1]] and w.tolist() == [[0.0, 0.0], [1.0, 0.0]]


@pytest.mark.parametrize("renorm", [False, True])
def test_route_and_gradient_against_torch(renorm):
    x = torch.from_numpy(np.random.default_rng(3).normal(size=(9, 17))).requires_grad_()
    p = torch.softmax(x, -1)
    v, i = torch.topk(p, 5)
    w = v / v.sum(-1, keepdim=True) if renorm else v
    idx, got = L.route(x.detach().numpy(), 5, renorm)
    assert np.array_equal(idx, i.numpy()) and np.allclose(got, w.detach().numpy(), rtol=1e-13)
    dw = torch.from_numpy(np.random.default_rng(4).normal(size=(9, 5)))
    w.backward(dw)
    assert np.allclose(L.route_backward(x.detach().numpy(), idx, got, dw.numpy(), renorm), x.grad.numpy(), atol=1e-14)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activations_against_torch(act):
    z = torch.linspace(-6, 6, 241, dtype=torch.float64, requires_grad=True)
    f = {"none": lambda t: t * 1.0, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "silu": torch.nn.functional.silu}[act]
    y = f(z)
    y.sum().backward()
    v, s = L.activation(z.detach().numpy(), act)
    assert np.allclose(v, y.detach().numpy(), atol=1e-13) and np.allclose(s, z.grad.numpy(), atol=1e-13)


@pytest.mark.parametrize("act,gated", [("none", False), ("gelu", False), ("silu", True), ("none", True)])
def test_linear_gradient_against_differences(act, gated):
    rng = np.random.default_rng(5)
    rows, G, I, O, counts = 7, 3, 4, 3, [3, 0, 2]
    N = 2 * O if gated else O
    x, w, b = rng.normal(size=(rows, I)), rng.normal(size=(G, N, I)), rng.normal(size=(G, N))
    dout = rng.normal(size=(rows, O))
    z = L.linear(x, w, act, gated, b, None, counts)[1]
    dx, dw, db, _ = L.linear_backward(dout, x, w, z if act != "none" or gated else None, act, gated, counts)
    f = lambda: float((L.linear(x, w, act, gated, b, None, counts)[0] * dout)[:5].sum())  # noqa: E731
    for v, g in ((x, dx), (w, dw), (b, db)):
        for at in np.ndindex(*v.shape):
            keep, h = v[at], 1e-5
            v[at] = keep + h
            up = f()
            v[at] = keep - h
            down = f()
            v[at] = keep
            assert abs((up - down) / (2 * h) - g[at]) < 1e-8, at


def test_group_ranges():
    assert L.group_ranges([2, -1, 0, 5], 6) == [(0, 2), (2, 2), (2, 2), (2, 6)]


def test_moe_layer_is_the_weighted_sum_of_its_experts():
    rng = np.random.default_rng(6)
    N, H, I, E, K = 3, 5, 4, 6, 2
    x, r = rng.normal(size=(N, H)), rng.normal(size=(E, H))
    up, down, res = rng.normal(size=(E, 2 * I, H)), rng.normal(size=(E, H, I)), rng.normal(size=(N, H))
    out, idx, w = L.moe_layer(x, r, up, down, "silu", True, K, True, res)
    t = [torch.from_numpy(v) for v in (x, r, up, down, res)]
    for n in range(N):
        want = t[4][n].clone()
        for k in range(K):
            z = t[2][idx[n, k]] @ t[0][n]
            want += w[n, k] * (t[3][idx[n, k]] @ (torch.nn.functional.silu(z[:I]) * z[I:]))
        assert np.allclose(out[n], want.numpy(), atol=1e-13)
