"""Products of rows in 8 bits whose scales are far from one: where the result is a binary32 number, it comes out."""
import numpy as np
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import DT, HALF, STEP, Tensors
from rows_util import pack, q8_window, row_bytes

pytestmark = pytest.mark.gpu

# few rows; 64 x 64 tiles, straight into the LDS and by registers; 64 x 128 tiles by expert; 128 x 128 twice; 256 x 256
# tile after tile (496 tiles, the last row's and column's ragged)
CASES = [(1, 3, 1, 640, 40, 0), (1, 100, 1, 640, 200, 0), (1, 100, 1, 640, 200, 1), (2, 90, 3, 256, 320, 0),
         (1, 2100, 1, 256, 2050, 0), (1, 8300, 1, 256, 2100, 0), (1, 7900, 1, 256, 4090, 0)]


@pytest.mark.parametrize("dtype,gated", [("f32", False), ("bf16", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("R,rows,G,I,O,off", CASES)
def test_large_scales_beside_small_ones(R, rows, G, I, O, off, dtype, gated):  # noqa: E741
    import torch
    O = (O + 1) // 2 if gated else O  # noqa: E741
    N = 2 * O if gated else O
    say(f"linear q8: scales up to 2^120, R={R} rows={rows} G={G} I={I} O={O} {dtype} gated={gated} off={off}")
    rng = np.random.default_rng(rows + I)
    xv, wv = (rng.integers(-127, 128, size=s, dtype=np.int8) for s in ((R, rows, I), (R, G, N, I)))
    # a row's scale is up to 2^120 and a channel's down to 2^-96: their product lies in 2^-97 .. 2^41; gated, the first
    # half's channels have 2^-120 and less, so that the product of both halves is below 2^127 too
    xs = (rng.uniform(0.5, 1.0, size=(R, rows)) * 2.0 ** rng.choice([0, 1, 30, 100, 120], size=(R, rows))).astype(np.float32)
    ws = (rng.uniform(1.0, 2.0, size=(R, G, N)) * 2.0 ** rng.choice([-96, -90, -80], size=(R, G, N))).astype(np.float32)
    if gated:
        ws[..., :O] *= np.float32(2.0 ** -24)
        ws[..., O:] *= np.float32(2.0 ** -20)
    xs[0, 0] = -xs[0, 0]  # any number will do
    counts = None
    if G > 1:
        counts = np.full((R, G), rows // G - 1, np.int32)
    act = vr.VR_ACT_GATED if gated else vr.VR_ACT_NONE
    with Job(R) as job:
        x = q8_window(job, (rows, row_bytes(I)), pack(xv, xs), off=4 * off)[0]
        w = q8_window(job, (G, N, row_bytes(I)), pack(wv, ws), off=4 * off)[0]
        out, read = Tensors(job, dtype).put(shape=(rows, O), fill=5.0)
        vr.vr_linear_q8(job.comm, vr.vrLinearShape(DT[dtype], rows, G, I, O, act), x, w, out,
                        group_rows=None if counts is None else torch.from_numpy(counts).cuda())
        got = read()
        for r in range(R):
            at = 0
            for g, n in enumerate([rows] if counts is None else counts[r].tolist()):
                z = torch.from_numpy(xv[r, at:at + n]).cuda().double() @ torch.from_numpy(wv[r, g]).cuda().double().T
                z = z * torch.from_numpy(xs[r, at:at + n, None]).cuda().double() * torch.from_numpy(ws[r, g]).cuda().double()
                want = z[:, :O] * z[:, O:] if gated else z
                # each half: the sum's conversion and two products; their product; the output's rounding; what lies below
                # the normal numbers
                tol = want.abs() * ((7 if gated else 3) * STEP / 2 * 1.01 + HALF[dtype]) + 2.0 ** -126
                off_by = (torch.from_numpy(got[r, at:at + n]).cuda() - want).abs()
                assert bool((off_by <= tol).all()), (r, g, int((~(off_by <= tol)).sum()))
                at += n
            assert np.all(got[r, at:] == 5.0)
        job.assert_no_async_error()
