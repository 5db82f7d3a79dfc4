"""The layer operators at the sizes where they change form: few rows, small and
wide tiles, the router's lists at their fullest, the few-token layer's chunks."""
import numpy as np
import pytest

import collective_window_put_amd as vr
import test_gpu_linear
import test_gpu_moe_layer
import test_gpu_route
from gpu_util import Job, say
from layer_util import HALF, STEP, Tensors, check
from oracle import layers as L

pytestmark = pytest.mark.gpu

LINEAR = [  # R, rows, G, I, O, dtype, act, gated, bias, residual, off
    # few rows: one and two 16-row blocks, past them, contraction lengths of a few elements and of many steps
    (1, 2, 1, 5, 17, "bf16", "gelu", True, True, True, 0), (1, 17, 1, 4104, 40, "bf16", "silu", True, True, True, 0),
    (2, 32, 1, 1000, 31, "bf16", "gelu", False, True, True, 1), (1, 128, 1, 300, 50, "f32", "silu", False, True, True, 0),
    (1, 33, 1, 513, 30, "f32", "gelu", True, True, False, 1), (2, 60, 4, 264, 40, "bf16", "silu", True, True, True, 0),
    # 64 x 64 tiles: contraction lengths of one step, two, three, four and a remainder
    (1, 70, 1, 64, 72, "bf16", "gelu", False, True, True, 0), (1, 70, 1, 128, 136, "bf16", "silu", True, True, True, 0),
    (1, 129, 1, 192, 200, "bf16", "relu", False, False, True, 0), (1, 130, 1, 264, 72, "bf16", "gelu", True, True, False, 0),
    (1, 200, 1, 96, 136, "f32", "relu", False, True, True, 0), (1, 1200, 1, 72, 1048, "bf16", "silu", False, True, True, 0),
    # 128 x 128 tiles, whole and ragged, with and without 16-byte rows
    (1, 2050, 1, 136, 2056, "bf16", "gelu", False, True, True, 0), (2, 1100, 3, 200, 1032, "bf16", "silu", True, True, True, 0),
    (1, 2049, 1, 33, 2047, "bf16", "silu", False, True, True, 1), (1, 2100, 1, 68, 2052, "f32", "relu", False, True, True, 0),
]


@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_linear(case):
    test_gpu_linear.test_linear_and_gradients(*case)


MOE = [  # R, T, E, K, H, I, dtype, act, gated, renorm, residual, off
    # inner axes of more than one staged chunk; column groups of 8, 4 and 2 blocks of 16
    (1, 3, 40, 4, 72, 1100, "bf16", "silu", True, True, True, 0), (1, 1, 16, 4, 1032, 600, "bf16", "gelu", True, True, True, 0),
    (1, 2, 16, 4, 136, 1030, "f32", "silu", True, True, False, 0), (1, 9, 64, 8, 2050, 40, "bf16", "silu", True, True, True, 1),
    (1, 5, 64, 8, 1032, 72, "bf16", "relu", False, True, False, 0), (2, 20, 2, 2, 520, 72, "bf16", "silu", True, True, True, 0),
    # the logits in a launch of their own
    (2, 2, 256, 8, 1032, 24, "bf16", "silu", True, True, True, 0), (1, 2, 520, 4, 514, 16, "f32", "silu", False, False, True, 1),
    # one token: no list of its entries; as many entries as experts
    (1, 1, 8, 8, 100, 36, "f32", "silu", True, False, True, 0), (8, 1, 8, 8, 72, 40, "bf16", "gelu", True, True, True, 0),
]


@pytest.mark.parametrize("case", MOE, ids=str)
def test_moe_layer(case):
    test_gpu_moe_layer.test_moe_layer(*case)


def test_moe_layer_one_token_of_nan():
    import torch
    say("moe layer: one NaN token")
    E, K, H, I = 8, 3, 64, 32  # noqa: E741
    d, router = test_gpu_moe_layer._data(1, 1, E, H, I, "bf16", True, 1)
    d["x"][0, 0, 5] = np.nan
    shape = vr.vrMoeShape(vr.VR_DT_BF16, 1, H, I, E, K, vr.VR_ACT_SILU | vr.VR_ACT_GATED, 0)
    need = vr.vr_moe_layer_workspace_bytes(1, shape)
    with Job(1) as job:
        tn = Tensors(job, "bf16")
        s = {k: tn.put(v)[0] for k, v in d.items()}
        out, read = tn.put(shape=(1, H), fill=5.0)
        idx = torch.zeros((1, 1, K), dtype=torch.int32, device="cuda")
        w = torch.ones((1, 1, K), device="cuda")
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        vr.vr_moe_layer(job.comm, shape, s["x"], torch.from_numpy(router).cuda().bfloat16(), s["w_up"], s["w_down"], out, idx, w,
                        residual=s["residual"], workspace=ws, workspace_bytes=need)
        assert np.array_equal(read(), d["residual"]) and (idx == -1).all() and not w.any()
        assert job.async_error()[1] == vr.VR_ASYNC_BAD_VALUE


ROUTE = [  # R, T, E, K, dtype, renorm, masked, levels, off
    (1, 5, 512, 16, "bf16", False, 0, None, 0), (2, 19, 500, 16, "f32", True, 0, 1, 1), (1, 3, 130, 16, "bf16", False, 120, 1, 3),
    (1, 16, 64, 16, "f32", False, 60, 2, 0), (3, 17, 33, 1, "bf16", True, 0, 2, 0), (1, 2, 17, 17, "f32", True, 5, None, 0),
    (1, 70, 200, 12, "bf16", True, 0, 3, 0), (1, 31, 16, 16, "bf16", False, 0, None, 1), (2, 4, 514, 3, "f32", False, 0, None, 0),
]


@pytest.mark.parametrize("case", ROUTE, ids=str)
def test_route(case):
    test_gpu_route.test_route_and_gradient(*case)


@pytest.mark.parametrize("E", [12, 256, 512])
def test_zeros_of_both_signs_tie_and_the_lowest_value_is_no_mask(E):
    import torch
    say(f"route: -0 and +0, the type's lowest value, E={E}")
    x = np.full((1, 2, E), -np.inf)
    x[0, 0, [3, 5, 7]] = [-0.0, 0.0, -0.0]
    x[0, 1, [2, 9]] = [np.finfo(np.float32).min, 1.0]
    with Job(1) as job:
        s, _ = Tensors(job, "f32").put(x)
        idx = torch.zeros((1, 2, 4), dtype=torch.int32, device="cuda")
        w = torch.zeros((1, 2, 4), device="cuda")
        vr.vr_route(job.comm, s, vr.VR_DT_F32, 2, 4, E, idx, w)
        assert idx[0].tolist() == [[3, 5, 7, -1], [9, 2, -1, -1]]
        check(w[0].double().cpu().numpy(), np.array([[1 / 3] * 3 + [0], [1, 0, 0, 0]]), 4 * STEP, "weights")
        job.assert_no_async_error()


@pytest.mark.parametrize("dtype,renorm", [("f32", False), ("bf16", False), ("f32", True)])
def test_gradient_of_entries_that_share_an_expert(dtype, renorm):
    import torch
    say(f"route backward: shared experts {dtype} renorm={renorm}")
    T, E, K = 9, 40, 6
    rng = np.random.default_rng(8)
    x = test_gpu_route._logits(1, T, E, dtype, 5)
    idx = rng.integers(0, 4, size=(1, T, K)).astype(np.int32)
    w, dw = (rng.random((1, T, K)).astype(np.float32) for _ in range(2))
    with Job(1) as job:
        tn = Tensors(job, dtype)
        s, _ = tn.put(x)
        ds, read = tn.put(shape=(T, E), fill=3.0)
        for _ in range(2):
            vr.vr_route_backward(job.comm, s, vr.VR_DT_F32 if dtype == "f32" else vr.VR_DT_BF16, T, K, E,
                                 torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(dw).cuda(), ds,
                                 vr.VR_ROUTE_RENORM if renorm else 0)
        want = L.route_backward(x, idx, w, dw, renorm)
        # K products and sums of values below K, exp and one division
        check(read(), want, np.abs(want) * HALF[dtype] + 2 * K * (np.abs(x).max() * 2 + 32 + K) * STEP, "dlogits")
        job.assert_no_async_error()
