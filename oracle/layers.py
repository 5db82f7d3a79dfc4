"""Plain definitions, in binary64, of the layers between the collectives: the
router, the linear layer (dense or by expert) and the few-token
mixture-of-experts layer, with their gradients, the root-mean-square norm, rows
in 8 bits and the combine's gradient.

Formulas (include/vrcomm.h states the same): softmax and its K largest; the
product x w^T + b with an activation, a gate and a residual; the layer as the
weighted sum of its experts. Pinned by tests/test_oracle_layers.py against
hand-worked cases, torch's functions and central differences.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["route", "route_backward", "activation", "linear", "linear_backward", "group_ranges", "moe_layer",
           "norm", "norm_backward", "to_8_bits", "combine_backward"]


def route(logits, K: int, renorm: bool):
    """(topk_idx int32, weights) of rows of logits: the K largest by falling
    logit, ties to the lowest index; -inf, +inf and NaN are never chosen."""
    x = np.asarray(logits, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    idx = np.full((flat.shape[0], K), -1, dtype=np.int32)
    w = np.zeros((flat.shape[0], K))
    for r, row in enumerate(flat):
        row = np.where(np.isfinite(row), row, -np.inf)
        if not np.isfinite(row).any():
            continue
        p = np.exp(row - row.max())
        order = [int(j) for j in np.argsort(-row, kind="stable") if row[j] > -np.inf][:K]
        part = p[order]
        idx[r, :len(order)] = order
        w[r, :len(order)] = part / (part.sum() if renorm else p.sum())
    return idx.reshape(*x.shape[:-1], K), w.reshape(*x.shape[:-1], K)


def route_backward(logits, topk_idx, weights, dweights, renorm: bool):
    """Gradient of the weights' inner product with dweights, for the routing topk_idx."""
    x = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(x)
    for at in np.ndindex(*x.shape[:-1]):
        e, w, d = topk_idx[at], np.asarray(weights[at], np.float64), np.asarray(dweights[at], np.float64)
        have = e >= 0
        mean = float((w[have] * d[have]).sum())
        if renorm:
            for k in np.flatnonzero(have):
                out[at][e[k]] += w[k] * (d[k] - mean)
            continue
        row = np.where(np.isfinite(x[at]), x[at], -np.inf)
        if not np.isfinite(row).any():
            continue
        p = np.exp(row - row.max())
        p /= p.sum()
        g = np.zeros_like(p)
        for k in np.flatnonzero(have):
            g[e[k]] += d[k]
        out[at] = p * (g - mean)
    return out


def activation(z, act: str):
    """(act(z), act'(z))."""
    from scipy.special import erf
    if act == "none":
        return z, np.ones_like(z)
    if act == "relu":
        return np.where(z > 0, z, 0.0), np.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        cdf = 0.5 * (1.0 + erf(z / math.sqrt(2.0)))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def group_ranges(counts, rows: int):
    """[first, last) of each group's rows: in order, negative counts as 0, cut at `rows`."""
    at, got = 0, []
    for c in counts:
        end = min(rows, at + max(0, int(c)))
        got.append((at, end))
        at = end
    return got


def linear(x, w, act: str, gated: bool, bias=None, residual=None, counts=None):
    """(out, z) of one rank: x [rows][I], w [G][N][I]; rows that no group holds are zero."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    G, N, _ = w.shape
    O = N // 2 if gated else N
    z, out = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], O))
    for g, (a, b) in enumerate(group_ranges([x.shape[0]] if counts is None else counts, x.shape[0])):
        z[a:b] = x[a:b] @ w[g].T + (0.0 if bias is None else np.asarray(bias, np.float64)[g])
        y = activation(z[a:b, :O], act)[0] * (z[a:b, O:] if gated else 1.0)
        out[a:b] = y + (0.0 if residual is None else np.asarray(residual, np.float64)[a:b])
    return out, z


def linear_backward(dout, x, w, z, act: str, gated: bool, counts=None):
    """(dx, dw, dbias, dz) of one rank."""
    dout, x, w = (np.asarray(v, np.float64) for v in (dout, x, w))
    G, N, _ = w.shape
    O = N // 2 if gated else N
    dx, dw, db, dz = np.zeros_like(x), np.zeros_like(w), np.zeros((G, N)), np.zeros((x.shape[0], N))
    for g, (a, b) in enumerate(group_ranges([x.shape[0]] if counts is None else counts, x.shape[0])):
        if z is None:
            dz[a:b] = dout[a:b]
        else:
            v = np.asarray(z, np.float64)[a:b]
            y, slope = activation(v[:, :O], act)
            dz[a:b] = np.concatenate([dout[a:b] * v[:, O:] * slope, dout[a:b] * y], 1) if gated else dout[a:b] * slope
        dx[a:b] = dz[a:b] @ w[g]
        dw[g] = dz[a:b].T @ x[a:b]
        db[g] = dz[a:b].sum(0)
    return dx, dw, db, dz


def moe_layer(x, router, w_up, w_down, act: str, gated: bool, K: int, renorm: bool, residual=None):
    """(out, topk_idx, weights): x [N][H], router [E][H], w_up [E][U][H], w_down [E][H][I]."""
    x, router, w_up, w_down = (np.asarray(v, np.float64) for v in (x, router, w_up, w_down))
    idx, weights = route(x @ router.T, K, renorm)
    out = np.zeros_like(x)
    I = w_down.shape[2]
    for n in range(x.shape[0]):
        for k in range(K):
            e = idx[n, k]
            if e < 0:
                continue
            z = w_up[e] @ x[n]
            h = activation(z[:I], act)[0] * (z[I:] if gated else 1.0)
            out[n] += weights[n, k] * (w_down[e] @ h)
    return out + (0.0 if residual is None else np.asarray(residual, np.float64)), idx, weights


def norm(h, gain, eps: float):
    """h / sqrt(mean h^2 + eps) * gain, row by row."""
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * (1.0 if gain is None else np.asarray(gain, np.float64))


def norm_backward(dout, h, gain, eps: float, dsum=None):
    """(dh, dgain) of rows h; dsum is what reaches h by other ways."""
    dout, h = np.asarray(dout, np.float64), np.asarray(h, np.float64)
    root = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, g = h / root, dout * (1.0 if gain is None else np.asarray(gain, np.float64))
    dh = (g - n * (g * n).mean(-1, keepdims=True)) / root
    return dh + (0.0 if dsum is None else np.asarray(dsum, np.float64)), (dout * n).sum(0)


def to_8_bits(x):
    """(int8 values, binary32 scales) of rows of binary32 values, bit for bit: scale m / 127 and the multiplier 127 / m
    rounded to binary32, the product rounded once; zeros below 2^-119, scale NaN where a value is no number. The largest
    number's scale is rounded down: 127 times it is a number."""
    x = np.asarray(x, np.float32)
    m = np.abs(x).max(-1, keepdims=True)
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    none = bad | (m < np.float32(2.0 ** -119))
    m1 = np.where(none, np.float32(1), m).astype(np.float32)
    most = np.nextafter(np.finfo(np.float32).max / np.float32(127), np.float32(0))
    value = np.rint(np.where(none, 0, x).astype(np.float64) * (np.float32(127) / m1).astype(np.float64))
    scale = np.where(bad, np.float32(np.nan), np.where(none, np.float32(0), np.minimum(m1 / np.float32(127), most)))
    return value.astype(np.int8), scale[..., 0].astype(np.float32)


def combine_backward(dout, y, rank, row, weights):
    """(rows of dy that an entry names, as {(rank, row): gradient}, dweights) of dout [S][T][H], y [R][rows][H]; rank and
    row [S][T][K] name an entry's row, -1 for none."""
    dy, dw = {}, np.zeros(np.shape(weights))
    for at in np.ndindex(*dw.shape):
        d, p = int(rank[at]), int(row[at])
        if d >= 0 and p >= 0:
            dy[d, p] = float(weights[at]) * np.asarray(dout[at[:2]], np.float64)
            dw[at] = float(np.dot(np.asarray(dout[at[:2]], np.float64), np.asarray(y[d][p], np.float64)))
    return dy, dw
