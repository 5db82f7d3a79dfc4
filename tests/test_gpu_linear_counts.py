"""vr_linear and its gradients refuse counts that are no 32-bit words of memory, as the products of rows in 8 bits do."""
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import Tensors, workspace
from rows_util import refused

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [1, 3])
def test_counts_at_odd_addresses(groups):
    import torch
    say(f"linear: counts at odd addresses, groups={groups}")
    R, rows, n = 2, 6, 24
    shape = vr.vrLinearShape(vr.VR_DT_F32, rows, groups, n, n, 0)
    with Job(R) as job:
        tn = Tensors(job, "f32")
        x, w, out = tn.put(shape=(rows, n))[0], tn.put(shape=(groups * n, n))[0], tn.put(shape=(rows, n))[0]
        dx, dw, db = tn.put(shape=(rows, n))[0], tn.put(shape=(groups * n, n))[0], tn.put(shape=(groups, n))[0]
        counts = torch.zeros(R * groups + 1, dtype=torch.int32, device="cuda")
        need = vr.vr_linear_backward_workspace_bytes(R, shape)
        room = dict(workspace=workspace(need), workspace_bytes=need)
        for off in (1, 2, 3):
            at = counts.data_ptr() + off
            refused(lambda: vr.vr_linear(job.comm, shape, x, w, out, group_rows=at))
            refused(lambda: vr.vr_linear_backward(job.comm, shape, out, x, w, dx=dx, dw=dw, dbias=db, group_rows=at, **room))
        vr.vr_linear(job.comm, shape, x, w, out, group_rows=counts[1:])  # words, at any of them
        vr.vr_linear_backward(job.comm, shape, out, x, w, dx=dx, dw=dw, dbias=db, group_rows=counts[1:], **room)
        job.assert_no_async_error()
