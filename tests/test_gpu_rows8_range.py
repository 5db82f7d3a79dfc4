"""Rows in 8 bits whose largest magnitude is the type's largest number, as masks have it, come back as numbers."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, STEP, Tensors, round_to
from oracle import layers as L
from rows_util import pack, q8_window, row_bytes, unpack

LARGEST = {"f32": float(np.finfo(np.float32).max), "bf16": float.fromhex("0x1.fep127")}


def _rows(dtype, cols):
    x = round_to(np.random.default_rng(cols).normal(size=(1, 5, cols)), dtype)
    x[0, 0, 0] = -LARGEST[dtype]
    x[0, 1, cols - 1] = LARGEST[dtype]
    x[0, 2, cols // 2:] = -LARGEST[dtype]
    x[0, 3] = float(np.nextafter(np.float32(LARGEST["f32"]), np.float32(0))) if dtype == "f32" else LARGEST[dtype]
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_definition_stays_finite(dtype):
    x = _rows(dtype, 40)[0]
    values, scales = L.to_8_bits(x)
    back = values.astype(np.float32) * scales[:, None]
    assert np.isfinite(back).all()
    assert np.all(np.abs(back - x) <= scales[:, None].astype(np.float64) * (0.5 + 127 * 4 * STEP))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [3, 40, 600, 5000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_number_comes_back(dtype, cols):
    say(f"rows in 8 bits: the largest number, cols={cols} {dtype}")
    x = _rows(dtype, cols)
    with Job(1) as job:
        q8, read = q8_window(job, (5, row_bytes(cols)))
        vr.vr_quantize(job.comm, Tensors(job, dtype).put(x)[0], DT[dtype], 5, cols, q8)
        assert np.array_equal(read()[0], pack(*L.to_8_bits(x[0])))
        scales = unpack(read()[0], cols)[1].astype(np.float64)[:, None]
        wide, wide_read = Tensors(job, "f32").put(shape=(5, cols))
        vr.vr_dequantize(job.comm, q8, vr.VR_DT_F32, 5, cols, wide)
        got = wide_read()[0]
        assert np.isfinite(got).all() and np.all(np.abs(got - x[0]) <= scales * (0.5 + 127 * 4 * STEP))
        job.assert_no_async_error()
