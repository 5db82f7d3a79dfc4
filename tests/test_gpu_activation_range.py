"""Activations and their slopes over their whole range, relative to their own
size where they fall towards zero, and at infinities and NaN. The products are
zero and the bias is the argument, so nothing but the activation and its
rounding is between the argument and the output.

Bounds. bf16: one rounding, half a step (2^-8), and the evaluation, 2^-11 (the
upper tail of the normal distribution is held to 2.6e-4 of its value, 2^-11.9,
and the rest to a few binary32 steps). fp32: the argument of exp or erfc is
rounded once (half a step), which moves gelu's tail by z^2 / 2 steps more and
silu's by |z|; the functions and products take 16 steps. Slopes cross zero
between; there the bound is of their terms, below 2 each: 2^-19 (bf16: the tail
is held to 4.2e-7 absolutely) and 16 steps (fp32)."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import ACT, DT, HALF, STEP, Tensors, check, round_to, workspace
from scipy.special import log_ndtr

pytestmark = pytest.mark.gpu


def definition(z, act):
    """(act(z), act'(z)) in binary64, precise in both tails."""
    with np.errstate(invalid="ignore", over="ignore"):
        if act == "gelu":
            cdf = np.exp(log_ndtr(z))
            return z * cdf, cdf + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
        if act == "relu":
            return np.where(z > 0, z, np.where(np.isnan(z), z, 0.0)), np.where(z > 0, 1.0, 0.0)
        s = np.exp(-np.logaddexp(0.0, -z))
        return z * s, s * (1 + z * np.exp(-np.logaddexp(0.0, z)))


def relative(z, act, dtype):
    if dtype == "bf16":
        return HALF["bf16"] + 2.0 ** -11
    return HALF["f32"] + ((z * z / 2 if act == "gelu" else np.abs(z)) + 16) * STEP


def _run(job, z, rows, act, gated, dtype, I=8):  # noqa: E741
    """act(z) (gated: times 1) of a layer whose products are zero, on `rows` equal rows, and the bias' gradient of one row."""
    n = z.size
    bias = np.concatenate([z, np.ones(n)]) if gated else z
    tn = Tensors(job, dtype)
    code = ACT[act] | (vr.VR_ACT_GATED if gated else 0)
    shape = vr.vrLinearShape(DT[dtype], rows, 1, I, n, code)
    N = bias.size
    x, w = tn.put(shape=(rows, I))[0], tn.put(shape=(1, N, I))[0]
    b = tn.put(bias.reshape(1, 1, N))[0]
    out, read = tn.put(shape=(rows, n), fill=5.0)
    pre = tn.put(shape=(rows, N), fill=5.0)[0]
    vr.vr_linear(job.comm, shape, x, w, out, bias=b, preact=pre)
    got = read()[0]
    one = vr.vrLinearShape(DT[dtype], 1, 1, I, n, code)
    need = vr.vr_linear_backward_workspace_bytes(1, one)
    db, db_read = tn.put(shape=(1, N), fill=5.0)
    vr.vr_linear_backward(job.comm, one, tn.put(shape=(1, n), fill=1.0)[0], x, w, preact=pre, dbias=db,
                          workspace=workspace(need), workspace_bytes=need)
    return got, db_read()[0, 0]


@pytest.mark.parametrize("rows,gated", [(1, False), (1, True), (200, False), (70, True)])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_whole_range(dtype, act, rows, gated):
    say(f"activation range: {dtype} {act} rows={rows} gated={gated}")
    z = np.unique(round_to(np.concatenate([np.linspace(-12.0, 12.0, 1501), [-2.0 ** -40, 0.0, 2.0 ** -40, -0.7518, -1.2785]]), dtype))
    y, slope = definition(z, act)
    with Job(1) as job:
        got, db = _run(job, z, rows, act, gated, dtype)
        rel = relative(z, act, dtype)
        for r in {0, rows // 2, rows - 1}:
            check(got[r], y, np.abs(y) * rel, f"act row {r}")
        small = 2.0 ** -19 if dtype == "bf16" else 16 * STEP
        near = np.where(np.abs(z) < 3, small, 0.0)  # beyond, one term of the slope is much the larger
        check(db[:z.size], slope, np.abs(slope) * (rel + 4 * STEP) + near, "slope")
        if gated:  # the gradient of the second half is act(z)
            check(db[z.size:], y, np.abs(y) * rel, "gate's value")
        job.assert_no_async_error()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_few_token_layer_over_the_range(act):
    # x is the first unit vector, so w_up's first column is the argument; w_down is the identity, one expert of weight 1
    import torch
    say(f"activation range: few-token layer {act}")
    z = round_to(np.linspace(-12.0, 12.0, 512), "bf16")
    n = z.size
    for T in (1, 3):
        x, up = np.zeros((1, T, n)), np.zeros((1, 1, n, n))
        x[..., 0], up[0, 0, :, 0] = 1.0, z
        shape = vr.vrMoeShape(vr.VR_DT_BF16, T, n, n, 1, 1, ACT[act], vr.VR_ROUTE_RENORM)
        need = vr.vr_moe_layer_workspace_bytes(1, shape)
        with Job(1) as job:
            tn = Tensors(job, "bf16")
            out, read = tn.put(shape=(T, n), fill=5.0)
            idx = torch.zeros((1, T, 1), dtype=torch.int32, device="cuda")
            w = torch.zeros((1, T, 1), device="cuda")
            vr.vr_moe_layer(job.comm, shape, tn.put(x)[0], torch.zeros(1, n, device="cuda").bfloat16(), tn.put(up)[0],
                            tn.put(np.eye(n).reshape(1, 1, n, n))[0], out, idx, w, workspace=workspace(need), workspace_bytes=need)
            y, _ = definition(z, act)
            for t in range(T):  # 2^-16: held as two bf16 parts
                check(read()[0, t], y, np.abs(y) * (relative(z, act, "bf16") + 2.0 ** -16), f"token {t} of {T}")
            job.assert_no_async_error()


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan_as_in_the_definition(dtype, act):
    # z cdf(z) and z / (1 + exp(-z)) at -inf are -inf * 0, NaN, in both types
    say(f"activation of infinities: {dtype} {act}")
    z = np.array([-np.inf, np.inf, np.nan, -1e38, 1e38, -200.0, 200.0, -14.0, 14.0, 0.0, 1.0])
    z = round_to(z, dtype)
    y, _ = definition(z, act)
    for rows in (1, 200):
        with Job(1) as job:
            got, _ = _run(job, z, rows, act, False, dtype)
            for r in (0, rows - 1):
                assert np.array_equal(np.isnan(got[r]), np.isnan(y)), (got[r], y)
                fin = np.isfinite(y)
                assert np.array_equal(got[r][~fin & ~np.isnan(y)], y[~fin & ~np.isnan(y)])
                check(got[r][fin], y[fin], np.abs(y[fin]) * relative(np.clip(z[fin], -14, 14), act, dtype) + 2.0 ** -125, "finite")
