"""Refusals of the layer operators beside those in each operator's own tests."""
import pytest

import collective_window_put_amd as vr
from gpu_util import Job, say
from layer_util import Tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", ["first", "last"])
def test_group_counts_inside_the_workspace(at):
    # the gradient of z goes to the workspace, over counts that later launches read
    import torch
    say(f"linear backward: counts in the workspace's {at} bytes")
    R, rows, G, I, O = 2, 40, 3, 16, 8
    shape = vr.vrLinearShape(vr.VR_DT_F32, rows, G, I, O, vr.VR_ACT_RELU)
    need = vr.vr_linear_backward_workspace_bytes(R, shape)
    n = R * G * 4
    with Job(R) as job:
        tn = Tensors(job, "f32")
        dout, pre = tn.put(shape=(rows, O), fill=1.0)[0], tn.put(shape=(rows, O), fill=1.0)[0]
        x, w, dx = tn.put(shape=(rows, I))[0], tn.put(shape=(G, O, I))[0], tn.put(shape=(rows, I))[0]
        room = torch.zeros(need + 1024, dtype=torch.uint8, device="cuda")

        def call(counts):
            counts.fill_(10)
            vr.vr_linear_backward(job.comm, shape, dout, x, w, preact=pre, dx=dx, group_rows=counts, workspace=room,
                                  workspace_bytes=need)

        first = 0 if at == "first" else need - 4
        with pytest.raises(vr.VrError) as e:
            call(room[first:first + n].view(torch.int32))
        assert e.value.code == vr.VR_ERR_INVALID_ARGUMENT
        call(room[need:need + n].view(torch.int32))  # right behind it
        job.assert_no_async_error()
