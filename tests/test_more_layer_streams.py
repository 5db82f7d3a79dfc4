"""The norm, rows in 8 bits, their product and the combine's gradient on another stream and in a captured graph,
together as a block runs them. Outputs are overwritten before each run."""
import pytest

import collective_window_put_amd as vr
from gpu_util import ALIGN, Job, say
from test_layer_streams import Layer, assert_writes

pytestmark = pytest.mark.gpu


class More(Layer):
    def rows8(self, *shape, cols):
        """A window of rows in 8 bits, an output."""
        n = self.torch.Size(shape).numel() * vr.vr_q8_row_bytes(cols)
        h, views = self.job.window(max(ALIGN, n), fill=0)
        self.outs.extend(v[:n] for v in views)
        return vr.vrSlice(h, 0)

    def _norm(self, rows, cols):
        R, c = self.job.R, self.job.comm
        shape = vr.vrNormShape(self.dt, rows, cols, 1e-5)
        x, res, gain = self.window((rows, cols), 1.0), self.window((rows, cols), 1.0), self.window((cols,), 1.0)
        dout, dsum = self.window((rows, cols), 1.0), self.window((rows, cols), 1.0)
        total, out, dh, dg = self.window((rows, cols)), self.window((rows, cols)), self.window((rows, cols)), self.window((cols,))
        q8 = self.rows8(rows, cols=cols)
        room = self.room(vr.vr_norm_backward_workspace_bytes(R, shape))

        def call(stream=None):
            vr.vr_norm(c, shape, x, gain=gain, residual=res, sum=total, out=out, q8=q8, stream=stream)
            vr.vr_norm_backward(c, shape, dout, total, gain=gain, dsum=dsum, dh=dh, dgain=dg, stream=stream, **room)
        self.call = call

    def _block8(self, rows, G, H, I, act):  # noqa: E741
        """Norm to 8 bits, the experts' two products in 8 bits."""
        R, c = self.job.R, self.job.comm
        N = 2 * I if act & vr.VR_ACT_GATED else I
        norm = vr.vrNormShape(self.dt, rows, H, 1e-5)
        up, down = vr.vrLinearShape(self.dt, rows, G, H, I, act), vr.vrLinearShape(self.dt, rows, G, I, H, vr.VR_ACT_NONE)
        x, w1, w2 = self.window((rows, H), 1.0), self.window((G * N, H), H ** -0.5), self.window((G * H, I), I ** -0.5)
        x8, w18, w28, h8 = self.rows8(rows, cols=H), self.rows8(G * N, cols=H), self.rows8(G * H, cols=I), self.rows8(rows, cols=I)
        h, out, wide = self.window((rows, I)), self.window((rows, H)), self.window((rows, H))
        counts = self.torch.full((R, G), rows // G, dtype=self.torch.int32, device="cuda") if G > 1 else None
        by = dict(groups=G, group_rows=counts)

        def call(stream=None):
            s = dict(stream=stream)
            vr.vr_quantize(c, w1, self.dt, G * N, H, w18, **s)
            vr.vr_quantize(c, w2, self.dt, G * H, I, w28, **s)
            vr.vr_norm(c, norm, x, q8=x8, **s)
            vr.vr_linear_q8(c, up, x8, w18, h, group_rows=counts, **s)
            vr.vr_quantize(c, h, self.dt, rows, I, h8, **by, **s)
            vr.vr_linear_q8(c, down, h8, w28, out, group_rows=counts, **s)
            vr.vr_dequantize(c, x8, self.dt, rows, H, wide, **by, **s)
        self.call = call

    def _combine(self, T, E, K, cols):
        R, c, torch = self.job.R, self.job.comm, self.torch
        cap = T * R * K
        d, y, dy = self.window((T, cols), 1.0), self.window((cap, cols), 1.0), self.window((cap, cols))
        topk = torch.randint(0, E, (R, T, K), generator=self.gen, device="cuda", dtype=torch.int32)
        rank = (topk // (E // R)).reshape(-1).long()
        pos = torch.empty(R * T * K, dtype=torch.int32, device="cuda")
        for r in range(R):
            at = rank == r
            pos[at] = torch.arange(int(at.sum()), dtype=torch.int32, device="cuda")
        w, dw = self.array(R, T, K, random=True), self.array(R, T, K, out=True)
        self.outs = [t for t in self.outs if t.shape != (cap, cols)]
        self.rows_of_dy = dy

        def call(stream=None):
            vr.vr_combine_backward(c, d, y, cap, cols * self.tt.itemsize, self.dt, topk, w, pos, T, K, E, dy=dy, dweights=dw,
                                   stream=stream)
        # every row that an entry names, as one output: rows of nobody are not written
        dy_t = [t for t in self.dy_views]
        for r in range(R):
            self.outs.append(dy_t[r][:int((rank == r).sum())])
        self.call = call

    def window(self, shape, random=0.0):
        s = super().window(shape, random)
        if not random:
            self.dy_views = self.outs[-self.job.R:]
        return s


LAYERS = [  # R, dtype, operator and its sizes
    (2, "bf16", ("norm", 37, 520)), (1, "f32", ("norm", 5, 77)), (1, "bf16", ("norm", 1, 4096)), (1, "bf16", ("norm", 3, 40000)),
    (2, "f32", ("norm", 700, 96)), (1, "bf16", ("block8", 1, 1, 256, 128, vr.VR_ACT_SILU | vr.VR_ACT_GATED)),
    (2, "f32", ("block8", 96, 3, 100, 72, vr.VR_ACT_GELU)), (1, "bf16", ("block8", 2048, 1, 136, 2048, vr.VR_ACT_RELU)),
    (4, "bf16", ("block8", 300, 5, 256, 200, vr.VR_ACT_SILU | vr.VR_ACT_GATED)),
    (2, "bf16", ("combine", 33, 8, 3, 256)), (1, "f32", ("combine", 5, 4, 9, 77)),
]


@pytest.mark.parametrize("R,dtype,kind", LAYERS, ids=str)
def test_another_stream(R, dtype, kind):
    import torch
    say(f"another stream: R={R} {dtype} {kind}")
    with Job(R) as job:
        layer = More(job, kind, dtype)
        layer.call()
        torch.cuda.synchronize()
        want = [t.cpu() for t in layer.outs]
        kept = [t.clone() for t in layer.ins]
        busy = torch.zeros(1 << 28, device="cuda")
        for given in (True, False):  # the stream as an argument, and as the current one
            st = torch.cuda.Stream()

            def run():
                for t in layer.ins:
                    t.zero_()
                torch.cuda.synchronize()
                with torch.cuda.stream(st):
                    for _ in range(8):  # a few milliseconds of work before the inputs are in place
                        busy.add_(1.0)
                    for t, k in zip(layer.ins, kept):
                        t.copy_(k)
                    if not given:
                        layer.call()
                if given:
                    layer.call(stream=st)
                st.synchronize()

            assert_writes(layer.outs, want, run, given)
        job.assert_no_async_error()


@pytest.mark.parametrize("R,dtype,kind", LAYERS, ids=str)
def test_graph_replays(R, dtype, kind):
    import torch
    say(f"graph replays: R={R} {dtype} {kind}")
    with Job(R) as job:
        layer = More(job, kind, dtype)
        layer.call()
        torch.cuda.synchronize()
        want = [t.cpu() for t in layer.outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            layer.call()

        def replay():
            graph.replay()
            torch.cuda.synchronize()

        for rep in range(4):
            assert_writes(layer.outs, want, replay, rep)
            if rep % 2:  # eager work between the replays
                assert_writes(layer.outs, want, lambda: (layer.call(), torch.cuda.synchronize()), "eager")
        # other inputs, the same graph: nothing of the first run is kept
        before = [t.clone() for t in layer.ins]
        for i, t in enumerate(layer.ins):
            t.copy_(t.flip(0) if t.shape[0] > 1 else t * 0.5)
        layer.call()
        torch.cuda.synchronize()
        other = [t.cpu() for t in layer.outs]
        assert any(not torch.equal(a, b) for a, b in zip(other, want))
        assert_writes(layer.outs, other, replay, "other inputs")
        for t, b in zip(layer.ins, before):
            t.copy_(b)
        assert_writes(layer.outs, want, replay, "the first inputs")
        job.assert_no_async_error()
        del graph


def test_two_calls_at_once():
    """Two gradients on two streams of two communicators, each with its own workspace, and shared inputs."""
    import torch
    say("two norm gradients at once")
    with Job(1) as a, Job(1) as b:
        la, lb = More(a, ("norm", 300, 1000), "bf16"), More(b, ("norm", 300, 1000), "bf16")
        for t, k in zip(lb.ins, la.ins):
            t.copy_(k)
        la.call()
        torch.cuda.synchronize()
        want = [t.cpu() for t in la.outs]
        sa, sb = torch.cuda.Stream(), torch.cuda.Stream()

        def both():
            for _ in range(5):
                la.call(stream=sa)
                lb.call(stream=sb)
            torch.cuda.synchronize()

        assert_writes(la.outs + lb.outs, want + want, both, "both")
        a.assert_no_async_error()
        b.assert_no_async_error()
