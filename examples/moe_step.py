"""A mixture-of-experts layer over R virtual ranks, as a program uses the library.

    python examples/moe_step.py

A training step over many tokens, forward

    vr_route -> vr_dispatch -> vr_linear (up, gated) -> vr_linear (down) -> vr_combine

and backward

    vr_combine_backward -> vr_linear_backward (down, up) -> vr_combine -> vr_route_backward

a decoding step over a few tokens, vr_moe_layer, with the same weights, and the
layer as the block of a model has it: behind a root-mean-square norm that takes
the residual stream along (vr_norm, vr_norm_backward), with the router's product,
and served in 8 bits

    vr_norm -> vr_linear, vr_route -> vr_dispatch -> vr_linear_q8 -> vr_quantize -> vr_linear_q8 -> vr_combine
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_window_put_amd as vr  # noqa: E402

ALIGN = vr.VR_WIN_REQUIRED_ALIGNMENT
DT = {torch.float32: vr.VR_DT_F32, torch.bfloat16: vr.VR_DT_BF16}


class Windows:
    """A communicator and windows of torch memory: one aligned slice per rank and tensor."""

    def __init__(self, R: int):
        self.R, self.comm = R, vr.vr_comm_create(R, signal_count=4)
        self.handles = []

    def tensor(self, shape, dtype):
        """(tensor [R, *shape], its vrSlice); the ranks' slices need not be adjacent."""
        n = torch.Size(shape).numel()
        size = n * dtype.itemsize
        stride = max(ALIGN, (size + ALIGN - 1) // ALIGN * ALIGN)
        slab = torch.zeros(self.R * stride + ALIGN, dtype=torch.uint8, device="cuda")
        shift = (-slab.data_ptr()) % ALIGN
        flat = slab[shift:shift + self.R * stride].view(dtype).view(self.R, -1)[:, :n]
        handle = vr.vr_window_register(self.comm, [flat[r].data_ptr() for r in range(self.R)], max(size, 1))
        self.handles.append(handle)
        return flat.unflatten(1, shape), vr.vrSlice(handle, 0)

    def close(self):
        torch.cuda.synchronize()
        for h in self.handles:
            vr.vr_window_deregister(self.comm, h)
        vr.vr_comm_destroy(self.comm)


class MoeStep:
    """The layer's tensors and workspaces for T tokens per rank of H elements, E experts of H -> I -> H, top-K."""

    def __init__(self, R, T, H, I, E, K, dtype=torch.bfloat16):  # noqa: E741
        self.R, self.T, self.H, self.I, self.E, self.K, self.dtype = R, T, H, I, E, K, dtype
        self.win = w = Windows(R)
        self.rows = rows = R * T * K  # no row is ever dropped
        G = E // R
        for name, shape in dict(x=(T, H), logits=(T, E), recv=(rows, H), preact=(rows, 2 * I), h=(rows, I), y=(rows, H),
                                out=(T, H), w_up=(G, 2 * I, H), w_down=(G, H, I), dout=(T, H), dy=(rows, H), dh=(rows, I),
                                drecv=(rows, H), dx=(T, H), dw_up=(G, 2 * I, H), dw_down=(G, H, I),
                                dlogits=(T, E)).items():
            t, s = w.tensor(shape, dtype)
            setattr(self, name, t)
            setattr(self, "_" + name, s)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.topk, self.pos = torch.empty(R, T, K, **i32), torch.empty(R, T, K, **i32)
        self.weights = torch.empty(R, T, K, device="cuda")
        self.counts, self.src = torch.empty(R, G, **i32), torch.empty(R, rows, **i32)
        dt = DT[dtype]
        self.up = vr.vrLinearShape(dt, rows, G, H, I, vr.VR_ACT_SILU | vr.VR_ACT_GATED)
        self.down = vr.vrLinearShape(dt, rows, G, I, H, vr.VR_ACT_NONE)
        need = max(vr.vr_linear_workspace_bytes(R, self.up), vr.vr_linear_workspace_bytes(R, self.down),
                   vr.vr_linear_backward_workspace_bytes(R, self.up), vr.vr_linear_backward_workspace_bytes(R, self.down))
        self.ws = dict(workspace=torch.empty(need, dtype=torch.uint8, device="cuda") if need else None, workspace_bytes=need)

    def _scatter(self, x, recv):
        vr.vr_dispatch(self.win.comm, x.window, 0, self.H * self.dtype.itemsize, self.topk, self.T, self.K, self.E, recv.window,
                       0, self.rows, self.counts, self.src, self.pos, 0, 1)

    def _gather(self, y, weights, out):
        vr.vr_combine(self.win.comm, y.window, 0, self.rows, self.H * self.dtype.itemsize, DT[self.dtype], self.topk, weights,
                      self.pos, self.T, self.K, self.E, out.window, 0, 2)

    def forward(self):
        """out from x and logits."""
        c = self.win.comm
        vr.vr_route(c, self._logits, DT[self.dtype], self.T, self.K, self.E, self.topk, self.weights, vr.VR_ROUTE_RENORM)
        self._scatter(self._x, self._recv)
        vr.vr_linear(c, self.up, self._recv, self._w_up, self._h, preact=self._preact, group_rows=self.counts, **self.ws)
        vr.vr_linear(c, self.down, self._h, self._w_down, self._y, group_rows=self.counts, **self.ws)
        self._gather(self._y, self.weights, self._out)

    def backward(self):
        """dx, dw_up, dw_down and dlogits from dout, after forward."""
        c, R, K = self.win.comm, self.R, self.K
        dweights = torch.empty_like(self.weights)
        vr.vr_combine_backward(c, self._dout, self._y, self.rows, self.H * self.dtype.itemsize, DT[self.dtype], self.topk,
                               self.weights, self.pos, self.T, K, self.E, dy=self._dy, dweights=dweights)
        vr.vr_linear_backward(c, self.down, self._dy, self._h, self._w_down, dx=self._dh, dw=self._dw_down,
                              group_rows=self.counts, **self.ws)
        vr.vr_linear_backward(c, self.up, self._dh, self._recv, self._w_up, preact=self._preact, dx=self._drecv,
                              dw=self._dw_up, group_rows=self.counts, **self.ws)
        self._gather(self._drecv, torch.ones_like(self.weights), self._dx)
        vr.vr_route_backward(c, None, DT[self.dtype], self.T, K, self.E, self.topk, self.weights, dweights, self._dlogits,
                             vr.VR_ROUTE_RENORM)

    def decode(self, tokens, router):
        """out [R, tokens, H] of the first `tokens` tokens of x on every rank, their experts and weights."""
        R, c = self.R, self.win.comm
        shape = vr.vrMoeShape(DT[self.dtype], tokens, self.H, self.I, self.E, self.K, vr.VR_ACT_SILU | vr.VR_ACT_GATED,
                              vr.VR_ROUTE_RENORM)
        need = vr.vr_moe_layer_workspace_bytes(R, shape)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        idx = torch.empty(R, tokens, self.K, dtype=torch.int32, device="cuda")
        weights = torch.empty(R, tokens, self.K, device="cuda")
        out, s = self.win.tensor((tokens, self.H), self.dtype)
        vr.vr_moe_layer(c, shape, self._x, router, self._w_up, self._w_down, s, idx, weights, workspace=ws, workspace_bytes=need)
        return out, idx, weights

    def check(self):
        torch.cuda.synchronize()
        code, bits = vr.vr_comm_get_async_error(self.win.comm)
        if code != vr.VR_OK:
            raise vr.VrError(code, f"asynchronous error bits {bits:#x}")

    def close(self):
        self.check()
        self.win.close()


class MoeBlock(MoeStep):
    """The layer behind a norm: stream = branch + residual, x = norm(stream) * gain, logits = x router^T, out = the layer's.
    The next block adds out to stream. Weights are kept in 8 bits too, for serving."""

    EPS = 1e-5

    def __init__(self, R, T, H, I, E, K, dtype=torch.bfloat16):  # noqa: E741
        super().__init__(R, T, H, I, E, K, dtype)
        G, rows = E // R, self.rows
        for name, shape in dict(branch=(T, H), residual=(T, H), stream=(T, H), gain=(H,), router=(1, E, H), dstream=(T, H),
                                dx_router=(T, H), dbranch=(T, H), dgain=(H,), drouter=(1, E, H)).items():
            t, s = self.win.tensor(shape, dtype)
            setattr(self, name, t)
            setattr(self, "_" + name, s)
        self.row_h, self.row_i = vr.vr_q8_row_bytes(H), vr.vr_q8_row_bytes(I)
        for name, shape in dict(x8=(T, self.row_h), recv8=(rows, self.row_h), h8=(rows, self.row_i),
                                w_up8=(G * 2 * I, self.row_h), w_down8=(G * H, self.row_i)).items():
            t, s = self.win.tensor(shape, torch.uint8)
            setattr(self, name, t)
            setattr(self, "_" + name, s)
        self.norm = vr.vrNormShape(DT[dtype], T, H, self.EPS)
        self.scores = vr.vrLinearShape(DT[dtype], T, 1, H, E, vr.VR_ACT_NONE)
        need = max(vr.vr_norm_backward_workspace_bytes(R, self.norm), vr.vr_linear_backward_workspace_bytes(R, self.scores))
        self.ws2 = dict(workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), workspace_bytes=need)

    def forward(self):
        """out and stream from branch and residual."""
        c = self.win.comm
        vr.vr_norm(c, self.norm, self._branch, gain=self._gain, residual=self._residual, sum=self._stream, out=self._x)
        vr.vr_linear(c, self.scores, self._x, self._router, self._logits)
        super().forward()

    def backward(self):
        """The layer's gradients, and dbranch (residual's is the same), dgain and drouter, from dout and dstream."""
        c = self.win.comm
        super().backward()
        vr.vr_linear_backward(c, self.scores, self._dlogits, self._x, self._router, dx=self._dx_router, dw=self._drouter,
                              **self.ws2)
        self.dx.add_(self.dx_router)
        vr.vr_norm_backward(c, self.norm, self._dx, self._stream, gain=self._gain, dsum=self._dstream, dh=self._dbranch,
                            dgain=self._dgain, **self.ws2)

    def quantize_weights(self):
        c, dt, G = self.win.comm, DT[self.dtype], self.E // self.R
        vr.vr_quantize(c, self._w_up, dt, G * 2 * self.I, self.H, self._w_up8)
        vr.vr_quantize(c, self._w_down, dt, G * self.H, self.I, self._w_down8)

    def serve(self):
        """out and stream in 8 bits: half the dispatch's bytes and the experts' weights'."""
        c, dt = self.win.comm, DT[self.dtype]
        vr.vr_norm(c, self.norm, self._branch, gain=self._gain, residual=self._residual, sum=self._stream, out=self._x,
                   q8=self._x8)
        vr.vr_linear(c, self.scores, self._x, self._router, self._logits)
        vr.vr_route(c, self._logits, dt, self.T, self.K, self.E, self.topk, self.weights, vr.VR_ROUTE_RENORM)
        vr.vr_dispatch(c, self._x8.window, 0, self.row_h, self.topk, self.T, self.K, self.E, self._recv8.window, 0, self.rows,
                       self.counts, self.src, self.pos, 0, 1)
        vr.vr_linear_q8(c, self.up, self._recv8, self._w_up8, self._h, group_rows=self.counts)
        vr.vr_quantize(c, self._h, dt, self.rows, self.I, self._h8, groups=self.E // self.R, group_rows=self.counts)
        vr.vr_linear_q8(c, self.down, self._h8, self._w_down8, self._y, group_rows=self.counts)
        self._gather(self._y, self.weights, self._out)


def main():
    gen = torch.Generator(device="cuda").manual_seed(0)
    R, T, H, I, E, K = 8, 512, 1024, 512, 64, 8  # noqa: E741
    step = MoeStep(R, T, H, I, E, K)

    def fill(t, scale=1.0):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda") * scale)

    fill(step.x), fill(step.dout), fill(step.w_up, H ** -0.5), fill(step.w_down, I ** -0.5)
    router = (torch.randn(E, H, generator=gen, device="cuda") * H ** -0.5).bfloat16()
    step.logits.copy_(step.x.float() @ router.float().t())
    step.forward()
    step.backward()
    few, _, _ = step.decode(4, router)
    step.check()
    print("training step: out", tuple(step.out.shape), "rms", float(step.out.float().square().mean().sqrt()))
    print("decoding step: out", tuple(few.shape), "rms", float(few.float().square().mean().sqrt()))
    step.close()

    block = MoeBlock(R, T, H, I, E, K)
    fill(block.branch), fill(block.residual), fill(block.dout), fill(block.dstream)
    fill(block.w_up, H ** -0.5), fill(block.w_down, I ** -0.5), fill(block.router, H ** -0.5)
    block.gain.fill_(1.0)
    block.forward()
    block.backward()
    block.check()
    whole = block.out.float().clone()
    print("block: out rms", float(whole.square().mean().sqrt()), "dgain rms", float(block.dgain.float().square().mean().sqrt()))
    block.quantize_weights()
    block.serve()
    block.check()
    print("block in 8 bits: off by", float((block.out.float() - whole).norm() / whole.norm()))
    block.close()


if __name__ == "__main__":
    main()
