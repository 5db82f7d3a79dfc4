"""Rows in 8 bits on the GPU: to them bit for bit as the definition has it, and back."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, Tensors, round_to
from oracle import layers as L
from rows_util import GUARD, pack, q8_window, refused, row_bytes, unpack

pytestmark = pytest.mark.gpu

CASES = [  # R, rows, cols, groups, dtype, off
    (1, 1, 1, 1, "f32", 0), (1, 1, 4, 1, "bf16", 0), (2, 3, 5, 1, "bf16", 1), (1, 9, 123, 1, "f32", 1), (1, 9, 124, 2, "bf16", 0),
    (1, 9, 125, 3, "bf16", 0), (3, 40, 256, 7, "f32", 0), (2, 100, 512, 70, "bf16", 0), (1, 17, 513, 1, "bf16", 3),
    (1, 5, 1000, 2, "f32", 0), (1, 7, 1024, 1, "bf16", 0), (2, 3, 1499, 1, "f32", 2), (1, 4, 2048, 1, "bf16", 0),
    (1, 3, 4099, 1, "bf16", 1), (1, 2, 8192, 1, "f32", 0), (1, 2, 16000, 1, "bf16", 0), (2, 2, 33001, 1, "bf16", 1),
    (1, 2, 20000, 1, "f32", 0),
]


@pytest.mark.parametrize("R,rows,cols,groups,dtype,off", CASES)
def test_to_8_bits_and_back(R, rows, cols, groups, dtype, off):
    import torch
    say(f"rows in 8 bits R={R} rows={rows} cols={cols} groups={groups} {dtype} off={off}")
    rng = np.random.default_rng(rows * cols)
    x = round_to(rng.normal(size=(R, rows, cols)) * 10.0 ** rng.uniform(-20, 20, size=(R, rows, 1)), dtype)
    x[:, 0] = round_to(np.arange(cols) % 255 - 127.0, dtype) * (1 if dtype == "f32" else 0.5)  # halves, whole numbers
    if rows > 2:
        x[:, 1] = 0
    counts, used = None, [rows] * R
    if groups > 1:
        c = rng.integers(0, max(1, 2 * rows // groups), size=(R, groups)).astype(np.int32)
        c[:, 0] = 0
        for r in range(R):
            while c[r].sum() > rows:
                c[r, rng.integers(0, groups)] //= 2
        used, counts = c.sum(1).tolist(), torch.from_numpy(c).cuda()
    with Job(R) as job:
        tn = Tensors(job, dtype, off)
        q8, read = q8_window(job, (rows, row_bytes(cols)), off=4 * off)
        vr.vr_quantize(job.comm, tn.put(x)[0], DT[dtype], rows, cols, q8, groups=groups, group_rows=counts)
        data = read()
        for r in range(R):
            n = used[r]
            values, scales = L.to_8_bits(x[r, :n])
            assert np.array_equal(data[r, :n], pack(values, scales)), r
            assert np.all(data[r, n:] == GUARD)  # rows of no group
        for back in ("f32", "bf16"):
            wide, wide_read = Tensors(job, back, off).put(shape=(rows, cols), fill=5.0)
            vr.vr_dequantize(job.comm, q8, DT[back], rows, cols, wide, groups=groups, group_rows=counts)
            got = wide_read()
            for r in range(R):
                values, scales = unpack(data[r, :used[r]], cols)
                want = (values.astype(np.float32) * scales[:, None]).astype(np.float32)  # one rounding
                assert np.array_equal(got[r, :used[r]], round_to(want, back)) and np.all(got[r, used[r]:] == 5.0)
        job.assert_no_async_error()


@pytest.mark.parametrize("cols", [3, 600, 5000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_that_are_no_numbers_and_the_smallest(cols, dtype):
    say(f"rows in 8 bits: NaN, infinities, subnormals, cols={cols} {dtype}")
    x = round_to(np.random.default_rng(1).normal(size=(1, 8, cols)), dtype)
    x[0, 1, cols - 1], x[0, 2, 0], x[0, 3, cols // 2] = np.nan, np.inf, -np.inf
    x[0, 4] *= 2.0 ** -140
    x[0, 5] = 2.0 ** -119 * np.sign(x[0, 5])
    x[0, 6] = x[0, 5] * (1 - 2.0 ** -8)
    x[0, 7, cols // 2] = 3.0e38
    x[0] = round_to(x[0], dtype)
    with Job(1) as job:
        q8, read = q8_window(job, (8, row_bytes(cols)))
        vr.vr_quantize(job.comm, Tensors(job, dtype).put(x)[0], DT[dtype], 8, cols, q8)
        assert job.async_error()[1] == vr.VR_ASYNC_BAD_VALUE
        values, scales = unpack(read()[0], cols)
        want, ws = L.to_8_bits(x[0])
        assert np.array_equal(values, want) and np.array_equal(scales, ws, equal_nan=True)
        assert not scales[4] and scales[5] and not scales[6] and not values[6].any() and np.all(np.abs(values[5]) == 127)
        wide, wide_read = Tensors(job, "f32").put(shape=(8, cols))
        vr.vr_dequantize(job.comm, q8, vr.VR_DT_F32, 8, cols, wide)
        assert np.isnan(wide_read()[0, 1:4]).all()  # nothing of such a row passes for a number
        job.assert_no_async_error()


def test_bytes_of_any_kind_widen():
    # -128 and bytes behind the values do no harm
    say("rows in 8 bits: any bytes")
    cols, rows = 253, 7
    rng = np.random.default_rng(4)
    data = rng.integers(0, 256, (1, rows, row_bytes(cols)), dtype=np.uint8)
    data[..., -4:] = rng.normal(size=(1, rows, 1)).astype(np.float32).view(np.uint8)
    with Job(1) as job:
        q8, _ = q8_window(job, data.shape[1:], data)
        wide, read = Tensors(job, "f32").put(shape=(rows, cols))
        vr.vr_dequantize(job.comm, q8, vr.VR_DT_F32, rows, cols, wide)
        scale = np.ascontiguousarray(data[0, :, -4:]).view(np.float32)
        assert np.array_equal(read()[0], (data[0, :, :cols].view(np.int8).astype(np.float32) * scale).astype(np.float64))


@pytest.mark.parametrize("counts,used", [([20, -3, 10, 40], 50), ([2 ** 31 - 1, 2 ** 31 - 1, 5, 0], 50), ([0, 0, 0, -1], 0)])
def test_group_counts_past_the_rows_and_negative(counts, used):
    import torch
    say(f"rows in 8 bits: bad group counts {counts}")
    rows, cols = 50, 20
    x = round_to(np.random.default_rng(1).normal(size=(1, rows, cols)), "f32")
    with Job(1) as job:
        q8, read = q8_window(job, (rows, row_bytes(cols)))
        c = torch.tensor([counts], dtype=torch.int32, device="cuda")
        vr.vr_quantize(job.comm, Tensors(job, "f32").put(x)[0], vr.VR_DT_F32, rows, cols, q8, groups=4, group_rows=c)
        assert job.async_error()[1] == vr.VR_ASYNC_CAPACITY
        assert np.array_equal(read()[0, :used], pack(*L.to_8_bits(x[0, :used]))) and np.all(read()[0, used:] == GUARD)
        wide, wide_read = Tensors(job, "f32").put(shape=(rows, cols), fill=5.0)
        full, _ = q8_window(job, (rows, row_bytes(cols)), pack(*L.to_8_bits(x)))
        vr.vr_dequantize(job.comm, full, vr.VR_DT_F32, rows, cols, wide, groups=4, group_rows=c)
        assert job.async_error()[1] == vr.VR_ASYNC_CAPACITY
        assert np.all(wide_read()[0, :used] != 5.0) and np.all(wide_read()[0, used:] == 5.0)


def test_refusals():
    import torch
    say("rows in 8 bits: refusals")
    R, rows, cols = 2, 6, 24
    with Job(R) as job:
        tn = Tensors(job, "f32")
        x = tn.put(shape=(rows, cols))[0]
        q8, _ = q8_window(job, (rows, row_bytes(cols)))
        counts = torch.zeros(R, 3, dtype=torch.int32, device="cuda")
        for name in ("vr_quantize", "vr_dequantize"):
            def call(a=x, dt=vr.VR_DT_F32, n=rows, c=cols, b=q8, name=name, **k):
                first, last = (a, b) if name == "vr_quantize" else (b, a)
                return lambda: getattr(vr, name)(job.comm, first, dt, n, c, last, **k)
            refused(call(dt=2))
            refused(call(n=-1))
            refused(call(n=(1 << 24) + 1))
            refused(call(c=0))
            refused(call(c=(1 << 20) + 1))
            refused(call(n=rows + 4096))
            refused(call(a=None))
            refused(call(b=None))
            refused(call(b=(q8.window, q8.offset + 2)))
            refused(call(a=(x.window, x.offset + 2)))
            refused(call(a=(q8.window, q8.offset), b=q8))
            refused(call(groups=3))                       # counts are missing
            refused(call(groups=0, group_rows=counts))
            refused(call(groups=1025, group_rows=counts))
            refused(call(groups=3, group_rows=counts.cpu()))
            call(n=0)()
            call(groups=3, group_rows=counts)()
            call()()
        job.assert_no_async_error()


def test_counts_at_odd_addresses():
    import torch
    say("rows in 8 bits, their product: counts that are no 32-bit words of memory")
    R, rows, cols = 2, 6, 24
    with Job(R) as job:
        x = Tensors(job, "f32").put(shape=(rows, cols))[0]
        q8, _ = q8_window(job, (rows, row_bytes(cols)))
        w, _ = q8_window(job, (cols, row_bytes(cols)))
        counts = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
        shape = vr.vrLinearShape(vr.VR_DT_F32, rows, 1, cols, cols, 0)
        for off in (1, 2, 3):
            at = counts.data_ptr() + off
            refused(lambda: vr.vr_quantize(job.comm, x, vr.VR_DT_F32, rows, cols, q8, group_rows=at))
            refused(lambda: vr.vr_dequantize(job.comm, q8, vr.VR_DT_F32, rows, cols, x, group_rows=at))
            refused(lambda: vr.vr_linear_q8(job.comm, shape, q8, w, x, group_rows=at))
        job.assert_no_async_error()
