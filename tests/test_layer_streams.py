"""The layer operators on a stream of their own and in a captured graph: every
output is overwritten before each run, so that a call which launches nothing,
drops a launch or ignores its stream is seen. test_what_the_check_sees shows on
the CPU that it is."""
import pytest

import collective_window_put_amd as vr
from gpu_util import ALIGN, Job, say


def blank(outs):
    """Values that no operator here writes."""
    for t in outs:
        t.fill_(77)


def assert_writes(outs, want, run, what):
    """run() brings every output from blank to what it was."""
    blank(outs)
    run()
    import torch
    for i, (t, w) in enumerate(zip(outs, want)):
        assert torch.equal(t.cpu(), w), (what, i)


def test_what_the_check_sees():
    import torch
    a, b, src = torch.zeros(3), torch.zeros(2, dtype=torch.int32), torch.arange(3.0)

    def whole():
        a.copy_(src)
        b.fill_(5)

    whole()
    want = [a.clone(), b.clone()]
    assert_writes([a, b], want, whole, "whole")
    for part in (lambda: None, lambda: a.copy_(src), lambda: b.fill_(5), lambda: (a.zero_(), b.fill_(5))):
        with pytest.raises(AssertionError):
            assert_writes([a, b], want, part, "part")


class Layer:
    """An operator's tensors on R ranks, and call(stream) that runs it with its gradient."""

    def __init__(self, job, kind, dtype):
        import torch
        self.job, self.torch = job, torch
        self.tt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
        self.dt = {"f32": vr.VR_DT_F32, "bf16": vr.VR_DT_BF16}[dtype]
        self.gen = torch.Generator(device="cuda").manual_seed(11)
        self.ins, self.outs = [], []
        getattr(self, "_" + kind[0])(*kind[1:])

    def window(self, shape, random=0.0):
        n = self.torch.Size(shape).numel()
        h, views = self.job.window(max(ALIGN, n * self.tt.itemsize), fill=0)
        ranks = [v.view(self.tt)[:n].view(shape) for v in views]
        for t in ranks:
            if random:
                t.copy_(self.torch.randn(shape, generator=self.gen, device="cuda") * random)
        (self.ins if random else self.outs).extend(ranks)
        return vr.vrSlice(h, 0)

    def array(self, *shape, dtype="f32", random=False, out=False):
        torch = self.torch
        t = torch.zeros(shape, dtype=torch.int32 if dtype == "i32" else torch.float32, device="cuda")
        if random:
            t.normal_(generator=self.gen)
        (self.ins if random else self.outs if out else []).append(t)
        return t

    def room(self, need):
        return dict(workspace=self.torch.empty(need, dtype=self.torch.uint8, device="cuda") if need else None, workspace_bytes=need)

    def _route(self, T, E, K, flags):
        R, c = self.job.R, self.job.comm
        x, d = self.window((T, E), 1.0), self.window((T, E))
        idx, w = self.array(R, T, K, dtype="i32", out=True), self.array(R, T, K, out=True)
        dw = self.array(R, T, K, random=True)

        def call(stream=None):
            vr.vr_route(c, x, self.dt, T, K, E, idx, w, flags, stream=stream)
            vr.vr_route_backward(c, x, self.dt, T, K, E, idx, w, dw, d, flags, stream=stream)
        self.call = call

    def _linear(self, rows, G, I, O, act):  # noqa: E741
        R, c = self.job.R, self.job.comm
        N = 2 * O if act & vr.VR_ACT_GATED else O
        shape = vr.vrLinearShape(self.dt, rows, G, I, O, act)
        x, w, b = self.window((rows, I), 1.0), self.window((G, N, I), I ** -0.5), self.window((G, N), 1.0)
        res, dout = self.window((rows, O), 1.0), self.window((rows, O), 1.0)
        out, pre, dx = self.window((rows, O)), self.window((rows, N)), self.window((rows, I))
        dw, db = self.window((G, N, I)), self.window((G, N))
        counts = None
        if G > 1:
            counts = self.torch.full((R, G), rows // G, dtype=self.torch.int32, device="cuda")
        room = self.room(vr.vr_linear_backward_workspace_bytes(R, shape))

        def call(stream=None):
            vr.vr_linear(c, shape, x, w, out, bias=b, residual=res, preact=pre, group_rows=counts, stream=stream)
            vr.vr_linear_backward(c, shape, dout, x, w, preact=pre, dx=dx, dw=dw, dbias=db, group_rows=counts, stream=stream,
                                  **room)
        self.call = call

    def _moe(self, T, E, K, H, I):  # noqa: E741
        R, c = self.job.R, self.job.comm
        shape = vr.vrMoeShape(self.dt, T, H, I, E, K, vr.VR_ACT_SILU | vr.VR_ACT_GATED, vr.VR_ROUTE_RENORM)
        x, up = self.window((T, H), 1.0), self.window((E // R, 2 * I, H), H ** -0.5)
        down, res, out = self.window((E // R, H, I), I ** -0.5), self.window((T, H), 1.0), self.window((T, H))
        router = self.array(E, H, random=True)
        if self.tt != router.dtype:
            router = self.ins[-1] = router.to(self.tt)
        idx, w = self.array(R, T, K, dtype="i32", out=True), self.array(R, T, K, out=True)
        room = self.room(vr.vr_moe_layer_workspace_bytes(R, shape))
        self.call = lambda stream=None: vr.vr_moe_layer(c, shape, x, router, up, down, out, idx, w, residual=res, stream=stream, **room)


LAYERS = [  # R, dtype, operator and its sizes
    (2, "f32", ("route", 37, 72, 5, vr.VR_ROUTE_RENORM)), (1, "bf16", ("route", 9, 600, 20, 0)), (2, "bf16", ("route", 1, 64, 4, 0)),
    (1, "bf16", ("linear", 3, 1, 200, 72, vr.VR_ACT_SILU)), (2, "bf16", ("linear", 200, 1, 96, 160, vr.VR_ACT_GELU)),
    (1, "f32", ("linear", 130, 1, 77, 45, vr.VR_ACT_RELU)), (2, "bf16", ("linear", 96, 3, 136, 72, vr.VR_ACT_SILU | vr.VR_ACT_GATED)),
    (1, "bf16", ("linear", 4096, 1, 136, 2048, vr.VR_ACT_GELU)), (1, "bf16", ("moe", 1, 16, 4, 136, 72)),
    (2, "bf16", ("moe", 3, 8, 3, 64, 32)), (1, "f32", ("moe", 4, 520, 8, 512, 24)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("R,dtype,kind", LAYERS, ids=str)
def test_another_stream(R, dtype, kind):
    import torch
    say(f"another stream: R={R} {dtype} {kind}")
    with Job(R) as job:
        layer = Layer(job, kind, dtype)
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


@pytest.mark.gpu
@pytest.mark.parametrize("R,dtype,kind", LAYERS, ids=str)
def test_graph_replays(R, dtype, kind):
    import torch
    say(f"graph replays: R={R} {dtype} {kind}")
    with Job(R) as job:
        layer = Layer(job, kind, dtype)
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
        for t in layer.ins:
            t.mul_(0.5)
        layer.call()
        torch.cuda.synchronize()
        halved = [t.cpu() for t in layer.outs]
        assert any(not torch.equal(a, b) for a, b in zip(halved, want))
        assert_writes(layer.outs, halved, replay, "other inputs")
        for t, b in zip(layer.ins, before):
            t.copy_(b)
        assert_writes(layer.outs, want, replay, "the first inputs")
        job.assert_no_async_error()
        del graph
