"""What a mixture-of-experts block needs beside its router, products and collectives, as measured cases: the
root-mean-square norm with the residual's addition (vr_norm, vr_norm_backward), rows in 8 bits with a scale each
(vr_quantize, vr_dequantize), the matrix product of such rows and such weights, dense or by expert (vr_linear_q8), and
the gradient of the combine (vr_combine_backward).

A row in 8 bits: its int8 values, zeros, and its fp32 scale in the last 4 of its bytes, a multiple of 128; it stands for
values * scale. Every tensor that lives in a window is made with one 4096-byte aligned slice per rank, so the plain form
and the library's calls read the same memory. Outputs that are held in 8 bits are widened to bf16 within the pass.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ALIGN = 4096
_EPS = 1e-5


# ---- cases --------------------------------------------------------------------------------
def listed():
    return [
        # the norm before one decoded token's layer
        dict(name="norm token", op="norm", R=1, rows=1, cols=4096, dtype="bf16", residual=True, quant=False),
        # a prefill step's norm before a dispatch in 8 bits: 8 ranks x 4096 tokens
        dict(name="norm q8 prefill", op="norm", R=8, rows=4096, cols=2048, dtype="bf16", residual=True, quant=True),
        # its gradient in training, the residual stream's own gradient added
        dict(name="norm grad", op="norm_backward", R=8, rows=2048, cols=4096, dtype="bf16", dsum=True),
        # full precision at odd sizes: rows that are no multiple of a vector
        dict(name="norm grad odd", op="norm_backward", R=3, rows=1001, cols=777, dtype="f32", dsum=False),
        # what the experts' first product leaves, in 8 bits for the second: ragged groups
        dict(name="quantize experts", op="quantize", R=4, rows=8192, G=8, cols=512, dtype="bf16"),
        # weights laid out for the products in 8 bits, from full precision, odd rows
        dict(name="quantize weights odd", op="quantize", R=2, rows=1499, G=1, cols=1001, dtype="f32"),
        # one decoded token through a dense layer in 8 bits: the weights' bandwidth
        dict(name="linear q8 token", op="linear", R=1, rows=1, G=1, I=4096, O=4096, dtype="bf16", act="silu", gated=False,
             bias=True, residual=True),
        # a prefill step's dense layer in 8 bits
        dict(name="linear q8 dense", op="linear", R=1, rows=8192, G=1, I=4096, O=4096, dtype="bf16", act="gelu", gated=False,
             bias=True, residual=True),
        # the experts' first product over the dispatch's rows: 8 ranks x 32 experts, top-8 of 4096 tokens
        dict(name="linear q8 experts", op="linear", R=8, rows=32768, G=32, I=512, O=512, dtype="bf16", act="silu", gated=True,
             bias=False, residual=False),
        # odd sizes, results in full precision
        dict(name="linear q8 odd", op="linear", R=2, rows=777, G=1, I=1001, O=1499, dtype="f32", act="relu", gated=False,
             bias=True, residual=False),
        # the combine's gradient in training: 8 ranks x 4096 tokens of 512 bytes, top-8 of 256 experts (the dispatch's workload)
        dict(name="combine grad", op="combine_backward", R=8, T=4096, E=256, K=8, cols=256, dtype="bf16", unrouted=0.0),
        # a short batch, odd rows, entries without an expert
        dict(name="combine grad odd", op="combine_backward", R=3, T=37, E=72, K=5, cols=77, dtype="f32", unrouted=0.2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "quantize", "linear", "linear", "combine_backward"])
    R = rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward", "quantize"):
        rows, cols = _log_int(rng, 1, 8192 // R), _log_int(rng, 32, 8192)
        if rng.random() < 0.5:  # the widths of real layers
            cols = (cols + 63) // 64 * 64
        if op == "norm":
            return dict(op=op, R=R, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7, quant=rng.random() < 0.5)
        if op == "norm_backward":
            return dict(op=op, R=R, rows=rows, cols=cols, dtype=dtype, dsum=rng.random() < 0.5)
        return dict(op=op, R=R, rows=rows, G=rng.choice([1, rng.randint(2, 32)]), cols=cols, dtype=dtype)
    if op == "combine_backward":
        E = R * max(1, _log_int(rng, 8, 512) // R)
        cols, K = _log_int(rng, 16, 4096), rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 4096)
        while R * T * K * cols > 1 << 26:
            T = max(1, T // 2)
        return dict(op=op, R=R, T=T, E=E, K=K, cols=cols, dtype=dtype, unrouted=rng.choice([0.0, 0.0, 0.1, 0.5]))
    G = rng.choice([1, 1, rng.randint(2, 16)])
    rows = _log_int(rng, 1, 8192 // R)
    I, O = _log_int(rng, 32, 4096), _log_int(rng, 32, 4096)
    if rng.random() < 0.5:
        I, O = (I + 63) // 64 * 64, (O + 63) // 64 * 64
    while R * rows * I * O > 8192 * 4096 * 1024 or R * G * I * O > 1 << 27:
        rows, I, O = max(1, rows // 2), max(32, I // 2), max(32, O // 2)
    return dict(op=op, R=R, rows=rows, G=G, I=I, O=O, dtype=dtype, act=rng.choice(["none", "relu", "gelu", "silu"]),
                gated=rng.random() < 0.4, bias=rng.random() < 0.5, residual=rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------------------
def _slab(R, shape, dtype):
    """A tensor [R, *shape] of zeros whose R slices start on window-aligned addresses."""
    esize = torch.empty(0, dtype=dtype).element_size()
    n = math.prod(shape)
    stride = max(_ALIGN, (n * esize + _ALIGN - 1) // _ALIGN * _ALIGN)
    buf = torch.zeros(R * stride + _ALIGN, dtype=torch.uint8, device="cuda")
    shift = (-buf.data_ptr()) % _ALIGN
    flat = buf[shift:shift + R * stride].view(dtype)
    inner = [math.prod(shape[i + 1:]) for i in range(len(shape))]
    return flat.as_strided((R, *shape), (stride // esize, *inner))


def _normal(gen, R, shape, dtype, scale=1.0):
    t = _slab(R, shape, dtype)
    for r in range(R):  # a rank at a time: the fp32 values of a large window need not exist at once
        t[r].copy_(torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale)
    return t


def _row_bytes(cols):
    return (cols + 4 + 127) // 128 * 128


def _q8(gen, R, lead, cols):
    """Random rows in 8 bits [R, *lead, row bytes], of values that are normal with a size of each row's own."""
    t = _slab(R, (*lead, _row_bytes(cols)), torch.uint8)
    for r in range(R):
        v = torch.randn((*lead, cols), generator=gen, device="cuda")
        s = v.abs().amax(-1, keepdim=True) / 127
        t[r, ..., :cols] = torch.round(v / s).to(torch.int8).view(torch.uint8)
        s = s * (torch.rand((*lead, 1), generator=gen, device="cuda") + 0.5)
        t[r, ..., -4:] = s.view(torch.uint8)
    return t


def _group_rows(R, G, rows, seed):
    """Rows of every group ([R][G], on the host): ragged, some groups empty, the last sixteenth of the rows unused."""
    gen = torch.Generator().manual_seed(seed * 7919 + 13)
    used = rows - rows // 16
    share = torch.rand(R, G, generator=gen) + 0.5
    share[torch.rand(R, G, generator=gen) < 0.08] = 0
    share[:, 0] += 0.25
    edge = torch.floor(torch.cumsum(share, 1) / share.sum(1, keepdim=True) * used + 0.5).to(torch.int64)
    edge[:, -1] = used
    return torch.diff(edge, dim=1, prepend=torch.zeros(R, 1, dtype=torch.int64)).clamp_(min=0)


def _routing(gen, case):
    """Experts of every token (distinct, some entries without one), their weights, and where the dispatch puts their rows:
    by expert, then source rank, then token."""
    R, T, E, K = case["R"], case["T"], case["E"], case["K"]
    idx = torch.rand(R, T, E, generator=gen, device="cuda").argsort(-1)[..., :K].to(torch.int32)
    idx[torch.rand(R, T, K, generator=gen, device="cuda") < case["unrouted"]] = -1
    weights = torch.softmax(torch.randn(R, T, K, generator=gen, device="cuda"), -1)
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True)[1]
    count = torch.bincount(key, minlength=E + 1)
    first = torch.cumsum(count, 0) - count
    own_rank = (torch.arange(E + 1, device="cuda") // (E // R)).clamp(max=R - 1) * (E // R)
    place = torch.empty_like(flat)
    place[order] = torch.arange(len(flat), device="cuda")
    pos = torch.where(flat < 0, -1, place - first[own_rank[key]])
    cap = case_rows(case)
    pos = torch.where(pos < cap, pos, -1)  # past the capacity: dropped
    return idx, weights, pos.reshape(R, T, K).to(torch.int32)


def case_rows(case):
    """Receive rows of a rank: an eighth more than its mean share."""
    n = case["T"] * case["K"]
    return n + n // 8 + 1


_comms = {}  # one communicator per rank count, as a program keeps one


class _Program:
    """What a program keeps beside its tensors to call the library: the communicator, a window for each tensor and a
    workspace. Lays nothing out and computes nothing."""

    def __init__(self, case, tensors):
        import collective_window_put_amd as vr
        self.vr = vr
        R, op = case["R"], case["op"]
        if R not in _comms:
            _comms[R] = vr.vr_comm_create(R)
        self.comm = _comms[R]
        self.windows = []
        for name, t in tensors.items():
            setattr(self, name, None if t is None else self._window(t))
        self.dtype = {"f32": vr.VR_DT_F32, "bf16": vr.VR_DT_BF16}[case["dtype"]]
        self.workspace, self.workspace_bytes = None, 0
        if op == "linear":
            act = {"none": vr.VR_ACT_NONE, "relu": vr.VR_ACT_RELU, "gelu": vr.VR_ACT_GELU, "silu": vr.VR_ACT_SILU}[case["act"]]
            self.shape = vr.vrLinearShape(self.dtype, case["rows"], case["G"], case["I"], case["O"],
                                          act | (vr.VR_ACT_GATED if case["gated"] else 0))
        elif op in ("norm", "norm_backward"):
            self.shape = vr.vrNormShape(self.dtype, case["rows"], case["cols"], _EPS)
            if op == "norm_backward":
                self.workspace_bytes = vr.vr_norm_backward_workspace_bytes(R, self.shape)
                self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device="cuda")

    def _window(self, t):
        vr = self.vr
        nbytes = max(1, t[0].numel()) * t.element_size()
        self.windows.append(vr.vr_window_register(self.comm, [t[r].data_ptr() for r in range(t.shape[0])], nbytes))
        return vr.vrSlice(self.windows[-1], 0)

    def __del__(self):
        for w in self.windows:
            self.vr.vr_window_deregister(self.comm, w)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, dt, op = case["R"], _DT[case["dtype"]], case["op"]
    arrays = {"group_rows": None}
    if case.get("G", 1) > 1:
        count = _group_rows(R, case["G"], case["rows"], seed)
        arrays["most"] = int(count.max())  # the padded form's capacity
        arrays["group_rows"] = count.to(device="cuda", dtype=torch.int32)
    if op in ("norm", "norm_backward"):
        rows, cols = case["rows"], case["cols"]
        gain = _normal(gen, R, (cols,), dt, 0.2)
        gain += 1
        tensors = {"gain": gain}
        if op == "norm":
            tensors["x"] = _normal(gen, R, (rows, cols), dt, 0.5)
            tensors["residual"] = _normal(gen, R, (rows, cols), dt, 2.0) if case["residual"] else None
            tensors["sum"] = _slab(R, (rows, cols), dt) if case["residual"] else None
            tensors["out"] = None if case["quant"] else _slab(R, (rows, cols), dt)
            tensors["q8"] = _slab(R, (rows, _row_bytes(cols)), torch.uint8) if case["quant"] else None
            tensors["wide"] = _slab(R, (rows, cols), torch.bfloat16) if case["quant"] else None
        else:
            tensors["h"] = _normal(gen, R, (rows, cols), dt, 2.0)
            tensors["dout"] = _normal(gen, R, (rows, cols), dt)
            tensors["dsum"] = _normal(gen, R, (rows, cols), dt) if case["dsum"] else None
            tensors["dh"], tensors["dgain"] = _slab(R, (rows, cols), dt), _slab(R, (cols,), dt)
    elif op == "quantize":
        rows, cols = case["rows"], case["cols"]
        tensors = {"x": _normal(gen, R, (rows, cols), dt), "q8": _slab(R, (rows, _row_bytes(cols)), torch.uint8),
                   "wide": _slab(R, (rows, cols), torch.bfloat16)}
    elif op == "linear":
        G, rows, I, O = case["G"], case["rows"], case["I"], case["O"]
        N = 2 * O if case["gated"] else O
        tensors = {"x": _q8(gen, R, (rows,), I), "w": _q8(gen, R, (G, N), I),
                   "bias": _normal(gen, R, (G, N), dt) if case["bias"] else None,
                   "residual": _normal(gen, R, (rows, O), dt) if case["residual"] else None, "out": _slab(R, (rows, O), dt)}
        tensors["w"][..., -4:] = (tensors["w"][..., -4:].contiguous().view(torch.float32) * I ** -0.5).view(torch.uint8)
    else:
        T, cols = case["T"], case["cols"]
        arrays["topk_idx"], arrays["weights"], arrays["send_pos"] = _routing(gen, case)
        arrays["dweights"] = torch.zeros(R, T, case["K"], device="cuda")
        tensors = {"dout": _normal(gen, R, (T, cols), dt), "y": _normal(gen, R, (case_rows(case), cols), dt),
                   "dy": _slab(R, (case_rows(case), cols), dt)}
    s = {"case": case, **tensors, **arrays}
    if own:
        s["program"] = _Program(case, tensors)
    return s


# ---- the plain form -------------------------------------------------------------------------
def _scale(rows8):
    return rows8[..., -4:].contiguous().view(torch.float32)


def _widen(rows8, cols):
    """The values that rows in 8 bits stand for, in fp32."""
    return rows8[..., :cols].view(torch.int8).float() * _scale(rows8)


def _in_8_bits(v):
    """v rounded to 8 bits with a scale for each row, as bf16 values."""
    s = v.abs().amax(-1, keepdim=True) / 127
    return (torch.round(v / torch.where(s > 0, s, 1.0)) * s).to(torch.bfloat16)


def _norm(s):
    case, dt = s["case"], s["x"].dtype
    h, got = s["x"].float(), {}
    if case["residual"]:
        got["sum"] = (h + s["residual"].float()).to(dt)
        h = got["sum"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS) * s["gain"].float()[:, None]
    if case["quant"]:
        got["q8"] = _in_8_bits(y)
    else:
        got["out"] = y.to(dt)
    return got


def _norm_backward(s):
    h, dout, dt = s["h"].float(), s["dout"].float(), s["h"].dtype
    inv = torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
    n = h * inv
    g = dout * s["gain"].float()[:, None]
    dh = inv * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dh = dh + s["dsum"].float()
    return {"dh": dh.to(dt), "dgain": (dout * n).sum(1).to(dt)}


def _used(s):
    """Which rows belong to a group, [R, rows, 1]."""
    k = torch.arange(s["case"]["rows"], device="cuda")
    return (k < s["group_rows"].sum(1, keepdim=True))[..., None]


def _quantize(s):
    v = _in_8_bits(s["x"].float())
    return v if s["group_rows"] is None else torch.where(_used(s), v, 0.0)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _padded(s):
    """Where each row of the padded groups [R, G, most] comes from, and which of them are rows at all."""
    count = s["group_rows"].long()
    first = torch.cumsum(count, 1) - count
    k = torch.arange(s["most"], device=count.device)
    real = k < count[..., None]
    return torch.where(real, first[..., None] + k, 0), real


def _by_group(s, t):
    """t [R, rows, n] as [R * G, rows of the group, n], padded with zeros (one group: as it is)."""
    if s["group_rows"] is None:
        return t
    at, real = _padded(s)
    R, G, most = at.shape
    got = torch.gather(t, 1, at.reshape(R, G * most, 1).expand(-1, -1, t.shape[2])).reshape(R, G, most, -1)
    return torch.where(real[..., None], got, 0.0).reshape(R * G, most, -1)


def _by_row(s, t):
    """The inverse; rows that no group holds are zero."""
    if s["group_rows"] is None:
        return t
    at, real = _padded(s)
    R, G, most = at.shape
    rows, n = s["case"]["rows"], t.shape[-1]
    out = torch.zeros(R, rows + 1, n, dtype=t.dtype, device=t.device)  # the last row takes the padding
    where = torch.where(real, at, rows).reshape(R, G * most, 1).expand(-1, -1, n)
    return out.scatter_(1, where, t.reshape(R, G * most, n))[:, :rows]


def _linear(s):
    case = s["case"]
    O, I = case["O"], case["I"]
    w = _widen(s["w"], I)
    z = torch.bmm(_by_group(s, _widen(s["x"], I)), w.reshape(-1, *w.shape[2:]).transpose(1, 2).contiguous())
    if s["bias"] is not None:
        z = z + s["bias"].float().reshape(-1, 1, z.shape[-1])
    z = _by_row(s, z)
    y = _act(z[..., :O], case["act"]) * z[..., O:] if case["gated"] else _act(z, case["act"])
    if case["residual"]:
        y = y + s["residual"].float()
    if s["group_rows"] is not None:  # rows that no group holds stay as they are: zero
        y = torch.where(_used(s), y, 0.0)
    return y.to(s["out"].dtype)


def _combine_backward(s):
    case, pos = s["case"], s["send_pos"].long()
    R, cap = case["R"], s["y"].shape[1]
    have = pos >= 0
    rank = s["topk_idx"].clamp(min=0).long() // (case["E"] // R)
    dout = s["dout"].float()[:, :, None]  # [R, T, 1, cols]
    y = s["y"][rank, pos.clamp(min=0)].float()  # [R, T, K, cols]
    dweights = torch.where(have, (dout * y).sum(-1), 0.0)
    dy = torch.zeros(R, cap + 1, case["cols"], dtype=s["y"].dtype, device="cuda")  # the last row takes entries without one
    dy[rank, torch.where(have, pos, cap)] = (s["weights"][..., None] * dout).to(dy.dtype)
    return {"dy": dy[:, :cap], "dweights": dweights}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"norm": _norm, "norm_backward": _norm_backward, "quantize": _quantize, "linear": _linear,
                "combine_backward": _combine_backward}[op](s)
    p = s["program"]
    vr = p.vr
    if op == "norm":
        vr.vr_norm(p.comm, p.shape, p.x, gain=p.gain, residual=p.residual, sum=p.sum, out=p.out, q8=p.q8)
        if case["quant"]:
            vr.vr_dequantize(p.comm, p.q8, vr.VR_DT_BF16, case["rows"], case["cols"], p.wide)
        got = {"sum": s["sum"]} if case["residual"] else {}
        return {**got, **({"q8": s["wide"]} if case["quant"] else {"out": s["out"]})}
    if op == "norm_backward":
        vr.vr_norm_backward(p.comm, p.shape, p.dout, p.h, gain=p.gain, dsum=p.dsum, dh=p.dh, dgain=p.dgain,
                            workspace=p.workspace, workspace_bytes=p.workspace_bytes)
        return {"dh": s["dh"], "dgain": s["dgain"]}
    if op == "quantize":
        vr.vr_quantize(p.comm, p.x, p.dtype, case["rows"], case["cols"], p.q8, groups=case["G"], group_rows=s["group_rows"])
        vr.vr_dequantize(p.comm, p.q8, vr.VR_DT_BF16, case["rows"], case["cols"], p.wide, groups=case["G"],
                         group_rows=s["group_rows"])
        return s["wide"]
    if op == "linear":
        vr.vr_linear_q8(p.comm, p.shape, p.x, p.w, p.out, bias=p.bias, residual=p.residual, group_rows=s["group_rows"])
        return s["out"]
    row_bytes = case["cols"] * s["y"].element_size()
    vr.vr_combine_backward(p.comm, p.dout, p.y, s["y"].shape[1], row_bytes, p.dtype, s["topk_idx"], s["weights"],
                           s["send_pos"], case["T"], case["K"], case["E"], dy=p.dy, dweights=s["dweights"])
    return {"dy": s["dy"], "dweights": s["dweights"]}


# ---- what a pass cannot do without -------------------------------------------------------------
def work(case):
    op, R = case["op"], case["R"]
    es = 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_backward"):
        n = R * case["rows"] * case["cols"]
        if op == "norm_backward":
            return {"bytes": (n * (4 if case["dsum"] else 3) + 2 * R * case["cols"]) * es, "flops": 10 * n}
        in_8 = 2 * (n + 4 * R * case["rows"]) + 2 * n  # written, read, and widened to bf16
        return {"bytes": (n * (3 if case["residual"] else 1) + R * case["cols"]) * es + (in_8 if case["quant"] else n * es),
                "flops": 4 * n}
    if op == "quantize":
        rows = case["rows"] - (case["rows"] // 16 if case["G"] > 1 else 0)
        n = R * rows * case["cols"]
        return {"bytes": n * es + 2 * (n + 4 * R * rows) + 2 * n, "flops": 4 * n}
    if op == "combine_backward":
        rows = R * case["T"]
        k = rows * case["K"] * (1 - case["unrouted"])
        return {"bytes": (rows + 2 * k) * case["cols"] * es + rows * case["K"] * 16, "flops": 3 * k * case["cols"]}
    G, rows, I, O = case["G"], case["rows"], case["I"], case["O"]
    N = 2 * O if case["gated"] else O
    used = rows - rows // 16 if G > 1 else rows
    w, b = R * min(G, used) * N * (I + 4), R * min(G, used) * N if case["bias"] else 0
    return {"bytes": R * used * (I + 4) + w + (R * used * O * (2 if case["residual"] else 1) + b) * es, "flops": 2 * R * used * N * I}


# ---- the definition in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "quantize": _exact_quantize, "linear": _exact_linear,
            "combine_backward": _exact_combine_backward}[case["op"]](s, case)


def _nearest_in_8_bits(v):
    """Row by row the nearest of 255 evenly spaced values from -max to max."""
    top = v.abs().max(-1, keepdim=True).values
    steps = torch.nan_to_num(v * (127 / top), nan=0.0)
    return steps.round() * top / 127


def _exact_norm(s, case):
    h, got = s["x"].double(), {}
    if case["residual"]:
        got["sum"] = h + s["residual"].double()
        h = got["sum"].to(s["x"].dtype).double()  # the norm is of what the residual stream holds
    root = (h.square().sum(-1) / case["cols"] + _EPS).sqrt()
    y = h / root[..., None] * s["gain"].double().unsqueeze(1)
    got["q8" if case["quant"] else "out"] = _nearest_in_8_bits(y) if case["quant"] else y
    return got


def _exact_norm_backward(s, case):
    """By the quotient's rule: y_j = gain_j h_j / r, dr/dh_i = h_i / (cols r)."""
    h, dy = s["h"].double(), s["dout"].double()
    r = (h.square().sum(-1, keepdim=True) / case["cols"] + _EPS).sqrt()
    weighted = dy * s["gain"].double().unsqueeze(1)
    dr = -(weighted * h).sum(-1, keepdim=True) / r.square()
    dh = weighted / r + dr * h / (case["cols"] * r)
    if case["dsum"]:
        dh += s["dsum"].double()
    return {"dh": dh, "dgain": (dy * h / r).sum(1)}


def _exact_quantize(s, case):
    got = _nearest_in_8_bits(s["x"].double())
    if s["group_rows"] is not None:
        for r, n in enumerate(s["group_rows"].sum(1).tolist()):
            got[r, n:] = 0
    return got


def _act64(v, name):
    if name == "gelu":
        one = torch.ones((), dtype=v.dtype, device=v.device)
        return v * torch.distributions.Normal(0 * one, one).cdf(v)
    if name == "silu":
        return v * torch.sigmoid(v)
    return v.clamp(min=0) if name == "relu" else v


def _exact_linear(s, case):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    I, O = case["I"], case["O"]
    for r in range(case["R"]):
        at = 0
        for g, n in enumerate([case["rows"]] if s["group_rows"] is None else s["group_rows"][r].tolist()):
            x, w = s["x"][r, at:at + n], s["w"][r, g]
            z = x[:, :I].view(torch.int8).double() @ w[:, :I].view(torch.int8).double().T  # whole numbers
            z = z * _scale(x).double() * _scale(w).double().T
            if case["bias"]:
                z += s["bias"][r, g].double()
            y = _act64(z[:, :O], case["act"])
            if case["gated"]:
                y = y * z[:, O:]
            if case["residual"]:
                y = y + s["residual"][r, at:at + n].double()
            out[r, at:at + n] = y
            at += n
    return out


def _exact_combine_backward(s, case):
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    per = case["E"] // case["R"]
    for k in range(case["K"]):
        source, token = torch.nonzero(s["send_pos"][..., k] >= 0, as_tuple=True)
        rank, row = s["topk_idx"][source, token, k].long() // per, s["send_pos"][source, token, k].long()
        d = s["dout"][source, token].double()
        dweights[source, token, k] = torch.linalg.vecdot(d, s["y"][rank, row].double())
        dy[rank, row] = d * s["weights"][source, token, k, None].double()
    return {"dy": dy, "dweights": dweights}
