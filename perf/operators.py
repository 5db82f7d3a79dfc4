"""The layers between the collectives, as measured cases: the router
(vr_route, vr_route_backward), the matrix product with bias, activation and
residual over a window's rows, dense or by expert (vr_linear,
vr_linear_backward), and the whole mixture-of-experts layer for a few tokens
(vr_moe_layer).

Every tensor that lives in a window is made with one 4096-byte aligned slice
per rank, so the plain form and the library's calls read the same memory.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ALIGN = 4096


# ---- cases --------------------------------------------------------------------------------
def listed():
    return [
        # the routing of one prefill step: 8 ranks x 4096 tokens, top-8 of 256 experts (the dispatch's workload)
        dict(name="route prefill", op="route", R=8, T=4096, E=256, K=8, dtype="f32", renorm=True, masked=0),
        # the routing of one decoded token
        dict(name="route token", op="route", R=1, T=1, E=64, K=4, dtype="bf16", renorm=True, masked=0),
        # its gradient in training, weights without renormalization
        dict(name="route grad", op="route_backward", R=8, T=4096, E=256, K=8, dtype="bf16", renorm=False, masked=0),
        # an odd token count, an expert count that fills no wave, experts masked out
        dict(name="route grad odd", op="route_backward", R=3, T=1001, E=72, K=5, dtype="f32", renorm=True, masked=9),
        # one decoded token through a dense layer: the weights' bandwidth
        dict(name="linear token", op="linear", R=1, rows=1, G=1, I=4096, O=4096, dtype="bf16", act="silu", gated=False,
             bias=True, residual=True),
        # a prefill step's dense layer
        dict(name="linear dense", op="linear", R=1, rows=8192, G=1, I=4096, O=4096, dtype="bf16", act="gelu", gated=False,
             bias=True, residual=True),
        # the experts' first product over the dispatch's rows: 8 ranks x 32 experts, 512-byte rows, top-8 of 4096 tokens
        dict(name="linear experts", op="linear", R=8, rows=32768, G=32, I=256, O=512, dtype="bf16", act="silu", gated=True,
             bias=False, residual=False),
        # full precision at odd sizes: rows that are no multiple of a vector
        dict(name="linear odd f32", op="linear", R=2, rows=777, G=1, I=1001, O=1499, dtype="f32", act="relu", gated=False,
             bias=True, residual=False),
        # a dense layer's gradients
        dict(name="linear grad dense", op="linear_backward", R=1, rows=4096, G=1, I=4096, O=4096, dtype="bf16", act="gelu",
             gated=False, bias=True),
        # the experts' gradients: ragged groups, a gated activation
        dict(name="linear grad experts", op="linear_backward", R=4, rows=8192, G=8, I=1024, O=512, dtype="bf16", act="silu",
             gated=True, bias=False),
        # one decoded token through a whole mixture-of-experts layer
        dict(name="moe token", op="moe", R=1, T=1, E=64, K=8, H=2048, I=1024, dtype="bf16", act="silu", gated=True,
             renorm=True, residual=True),
        # a decoding batch of 8 ranks x 4 tokens, top-8 of 256 experts
        dict(name="moe batch", op="moe", R=8, T=4, E=256, K=8, H=2048, I=512, dtype="bf16", act="silu", gated=True,
             renorm=True, residual=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "linear", "linear", "linear_backward", "moe"])
    R = rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    act, gated = rng.choice(["none", "relu", "gelu", "silu"]), rng.random() < 0.4
    if op in ("route", "route_backward"):
        E = R * max(1, _log_int(rng, 8, 512) // R)
        return dict(op=op, R=R, T=_log_int(rng, 1, 4096), E=E, K=rng.randint(1, min(16, E)), dtype=dtype,
                    renorm=rng.random() < 0.5, masked=rng.choice([0, 0, rng.randint(1, E - 1)]))
    if op == "moe":
        E = R * max(1, _log_int(rng, 4, 128) // R)
        H, I = _log_int(rng, 64, 2048), _log_int(rng, 32, 1024)
        while E * H * I > 1 << 27:
            I //= 2
        return dict(op=op, R=R, T=_log_int(rng, 1, 64 // R), E=E, K=rng.randint(1, min(8, E)), H=H, I=I, dtype=dtype,
                    act=act if act != "none" else "silu", gated=gated, renorm=rng.random() < 0.5, residual=rng.random() < 0.5)
    G = rng.choice([1, 1, rng.randint(2, 16)])
    rows = _log_int(rng, 1, 8192 // R)
    I, O = _log_int(rng, 32, 4096), _log_int(rng, 32, 4096)
    if rng.random() < 0.5:  # the widths of real layers
        I, O = (I + 63) // 64 * 64, (O + 63) // 64 * 64
    while R * rows * I * O > 8192 * 4096 * 1024 or R * G * I * O > 1 << 27:
        rows, I, O = max(1, rows // 2), max(32, I // 2), max(32, O // 2)
    case = dict(op=op, R=R, rows=rows, G=G, I=I, O=O, dtype=dtype, act=act, gated=gated, bias=rng.random() < 0.5)
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


# ---- inputs -------------------------------------------------------------------------------
def _slab(R, shape, dtype):
    """A tensor [R, *shape] whose R slices start on window-aligned addresses."""
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


def _group_rows(case, seed):
    """Rows of every group ([R][G], on the host): ragged, some groups empty, the last sixteenth of the rows unused."""
    R, G, rows = case["R"], case["G"], case["rows"]
    gen = torch.Generator().manual_seed(seed * 7919 + 13)
    used = rows - rows // 16
    share = torch.rand(R, G, generator=gen) + 0.5
    share[torch.rand(R, G, generator=gen) < 0.08] = 0
    share[:, 0] += 0.25
    edge = torch.floor(torch.cumsum(share, 1) / share.sum(1, keepdim=True) * used + 0.5).to(torch.int64)
    edge[:, -1] = used
    return torch.diff(edge, dim=1, prepend=torch.zeros(R, 1, dtype=torch.int64)).clamp_(min=0)


_comms = {}  # one communicator per rank count, as a program keeps one


class _Program:
    """What a program keeps beside its tensors to call the library: the communicator, a window for each tensor and a
    workspace. Lays nothing out and computes nothing."""

    def __init__(self, case, tensors, arrays):
        import collective_window_put_amd as vr
        self.vr = vr
        R = case["R"]
        if R not in _comms:
            _comms[R] = vr.vr_comm_create(R)
        self.comm = _comms[R]
        self.windows = []
        for name, t in tensors.items():
            setattr(self, name, None if t is None else self._window(t))
        for name, t in arrays.items():
            setattr(self, name, t)
        dt = {"f32": vr.VR_DT_F32, "bf16": vr.VR_DT_BF16}[case["dtype"]]
        act = 0
        if "act" in case:
            act = {"none": vr.VR_ACT_NONE, "relu": vr.VR_ACT_RELU, "gelu": vr.VR_ACT_GELU, "silu": vr.VR_ACT_SILU}[case["act"]]
            act |= vr.VR_ACT_GATED if case["gated"] else 0
        self.flags = vr.VR_ROUTE_RENORM if case.get("renorm") else 0
        self.dtype = dt
        need = 0
        if case["op"].startswith("linear"):
            self.shape = vr.vrLinearShape(dt, case["rows"], case["G"], case["I"], case["O"], act)
            need = (vr.vr_linear_workspace_bytes if case["op"] == "linear" else vr.vr_linear_backward_workspace_bytes)(R, self.shape)
        elif case["op"] == "moe":
            self.shape = vr.vrMoeShape(dt, case["T"], case["H"], case["I"], case["E"], case["K"], act, self.flags)
            need = vr.vr_moe_layer_workspace_bytes(R, self.shape)
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        self.workspace_bytes = need

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
    s = {"case": case}
    if op in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        logits = _normal(gen, R, (T, E), dt)
        if case["masked"]:  # experts that may not be chosen, others for each token
            order = torch.rand(R, T, E, generator=gen, device="cuda").argsort(-1)
            logits.masked_fill_(order < case["masked"], -math.inf)
        tensors = {"logits": logits}
        arrays = {"topk_idx": torch.zeros(R, T, K, dtype=torch.int32, device="cuda"),
                  "weights": torch.zeros(R, T, K, dtype=torch.float32, device="cuda")}
        if op == "route_backward":
            arrays["topk_idx"], arrays["weights"] = _route(logits, K, case["renorm"])
            arrays["dweights"] = torch.randn(R, T, K, generator=gen, device="cuda")
            tensors["dlogits"] = _slab(R, (T, E), dt)
    elif op == "moe":
        T, E, K, H, I = case["T"], case["E"], case["K"], case["H"], case["I"]
        up = 2 * I if case["gated"] else I
        tensors = {"x": _normal(gen, R, (T, H), dt), "w_up": _normal(gen, R, (E // R, up, H), dt, H ** -0.5),
                   "w_down": _normal(gen, R, (E // R, H, I), dt, I ** -0.5),
                   "residual": _normal(gen, R, (T, H), dt) if case["residual"] else None, "out": _slab(R, (T, H), dt)}
        arrays = {"router": (torch.randn(E, H, generator=gen, device="cuda") * H ** -0.5).to(dt),
                  "topk_idx": torch.zeros(R, T, K, dtype=torch.int32, device="cuda"),
                  "weights": torch.zeros(R, T, K, dtype=torch.float32, device="cuda")}
    else:
        G, rows, I, O = case["G"], case["rows"], case["I"], case["O"]
        N = 2 * O if case["gated"] else O
        arrays = {"group_rows": None}
        if G > 1:
            count = _group_rows(case, seed)
            s["most"] = int(count.max())  # the padded form's capacity
            arrays["group_rows"] = count.to(device="cuda", dtype=torch.int32)
        tensors = {"x": _normal(gen, R, (rows, I), dt), "w": _normal(gen, R, (G, N, I), dt, I ** -0.5),
                   "bias": _normal(gen, R, (G, N), dt) if case["bias"] else None}
        if op == "linear":
            tensors["residual"] = _normal(gen, R, (rows, O), dt) if case["residual"] else None
            tensors["out"] = _slab(R, (rows, O), dt)
        else:
            tensors["preact"] = None
            if case["act"] != "none" or case["gated"]:  # as the forward pass leaves it
                tensors["preact"] = _slab(R, (rows, N), dt)
                tensors["preact"].copy_(_preact({**s, **tensors, **arrays}))
            tensors["dout"] = _normal(gen, R, (rows, O), dt)
            tensors["dx"], tensors["dw"] = _slab(R, (rows, I), dt), _slab(R, (G, N, I), dt)
            tensors["dbias"] = _slab(R, (G, N), dt) if case["bias"] else None
    s.update(tensors)
    s.update(arrays)
    if own:
        s["program"] = _Program(case, tensors, arrays)
    return s


# ---- the plain form -------------------------------------------------------------------------
def _route(logits, K, renorm):
    """Softmax over the row, the K largest (ties to the lowest index); a -inf logit is never taken."""
    x = logits.float()
    top = x.amax(-1, keepdim=True)
    e = torch.where(x > -math.inf, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :K]
    taken = torch.gather(x, -1, order) > -math.inf
    part = torch.where(taken, torch.gather(e, -1, order), 0.0)
    whole = part.sum(-1, keepdim=True) if renorm else e.sum(-1, keepdim=True)
    return torch.where(taken, order, -1).to(torch.int32), torch.where(taken, part / whole, 0.0)


def _route_backward(logits, topk_idx, weights, dweights, renorm):
    at = topk_idx.clamp(min=0).long()
    dw = torch.where(topk_idx >= 0, dweights, 0.0)
    mean = (dw * weights).sum(-1, keepdim=True)
    d = torch.zeros(logits.shape, dtype=torch.float32, device=logits.device)
    if renorm:
        return d.scatter_add_(-1, at, weights * (dw - mean)).to(logits.dtype)
    x = logits.float()
    top = x.amax(-1, keepdim=True)
    e = torch.where(x > -math.inf, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return (p * (d.scatter_add_(-1, at, dw) - mean)).to(logits.dtype)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _padded(s):
    """Where each row of the padded groups [R, G, most] comes from, and which of them are rows at all."""
    count = s["group_rows"].long()
    first = torch.cumsum(count, 1) - count
    k = torch.arange(s["most"], device=count.device)
    real = k < count[..., None]
    return torch.where(real, first[..., None] + k, 0), real


def _rows_to_groups(s, t):
    """t [R, rows, n] in fp32 as [R * G, rows of the group, n], padded with zeros (one group: as it is)."""
    if s["group_rows"] is None:
        return t.float()
    at, real = _padded(s)
    R, G, most = at.shape
    got = torch.gather(t, 1, at.reshape(R, G * most, 1).expand(-1, -1, t.shape[2])).reshape(R, G, most, -1)
    return torch.where(real[..., None], got.float(), 0.0).reshape(R * G, most, -1)


def _groups_to_rows(s, t):
    """The inverse; rows that no group holds are zero."""
    if s["group_rows"] is None:
        return t
    at, real = _padded(s)
    R, G, most = at.shape
    rows, n = s["case"]["rows"], t.shape[-1]
    out = torch.zeros(R, rows + 1, n, dtype=t.dtype, device=t.device)  # the last row takes the padding
    where = torch.where(real, at, rows).reshape(R, G * most, 1).expand(-1, -1, n)
    return out.scatter_(1, where, t.reshape(R, G * most, n))[:, :rows]


def _weights(s):
    w = s["w"].float()
    return w.reshape(-1, *w.shape[2:])


def _preact(s):
    x = _rows_to_groups(s, s["x"])
    z = torch.bmm(x, _weights(s).transpose(1, 2).contiguous())
    if s["bias"] is not None:
        z = z + s["bias"].float().reshape(-1, 1, z.shape[-1])
    return _groups_to_rows(s, z)


def _linear(s):
    case = s["case"]
    z = _preact(s)
    O = case["O"]
    y = _act(z[..., :O], case["act"]) * z[..., O:] if case["gated"] else _act(z, case["act"])
    if case["residual"]:
        y = y + s["residual"].float()
    if s["group_rows"] is not None:  # rows that no group holds stay as they are: zero
        k = torch.arange(case["rows"], device=y.device)
        y = torch.where((k < s["group_rows"].sum(1, keepdim=True))[..., None], y, 0.0)
    return y.to(s["out"].dtype)


def _linear_backward(s):
    case = s["case"]
    dy, O, dt = s["dout"].float(), case["O"], s["dout"].dtype
    if s["preact"] is not None:
        z = s["preact"].float()
        if case["gated"]:
            g, u = z[..., :O], z[..., O:]
            dz = torch.cat([dy * u * _act_slope(g, case["act"]), dy * _act(g, case["act"])], -1)
        else:
            dz = dy * _act_slope(z, case["act"])
    else:
        dz = dy
    dz = _rows_to_groups(s, dz)
    dx = _groups_to_rows(s, torch.bmm(dz, _weights(s))).to(dt)
    dw = torch.bmm(dz.transpose(1, 2).contiguous(), _rows_to_groups(s, s["x"]))
    got = {"dx": dx, "dw": dw.reshape(s["w"].shape).to(dt)}
    if case["bias"]:
        got["dbias"] = dz.sum(1).reshape(s["bias"].shape).to(dt)
    return got


def _moe(s):
    case = s["case"]
    R, T, K, H, I = case["R"], case["T"], case["K"], case["H"], case["I"]
    x = s["x"].reshape(R * T, H)
    logits = x.double() @ s["router"].double().t()  # 64 bits: which expert is K-th is a border
    idx, weights = _route64(logits, K, case["renorm"])
    e = idx.reshape(-1).long()
    per = case["E"] // R
    up = s["w_up"][e // per, e % per].float()  # [pairs, up, H]
    xp = x.float().repeat_interleave(K, 0)[:, :, None]
    z = torch.bmm(up, xp)[..., 0]
    h = _act(z[:, :I], case["act"]) * z[:, I:] if case["gated"] else _act(z, case["act"])
    del up
    y = torch.bmm(s["w_down"][e // per, e % per].float(), h[:, :, None])[..., 0].reshape(R * T, K, H)
    out = (weights[..., None] * y).sum(1)
    if case["residual"]:
        out = out + s["residual"].reshape(R * T, H).float()
    return {"out": out.reshape(R, T, H).to(s["x"].dtype), "topk_idx": idx.reshape(R, T, K), "weights": weights.reshape(R, T, K)}


def _route64(logits, K, renorm):
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    order = torch.sort(logits, dim=-1, descending=True, stable=True)[1][..., :K]
    part = torch.gather(p, -1, order)
    return order.to(torch.int32), (part / (part if renorm else p).sum(-1, keepdim=True)).float()


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "route":
            return dict(zip(("topk_idx", "weights"), _route(s["logits"], case["K"], case["renorm"])))
        if op == "route_backward":
            return _route_backward(s["logits"], s["topk_idx"], s["weights"], s["dweights"], case["renorm"])
        return {"linear": _linear, "linear_backward": _linear_backward, "moe": _moe}[op](s)
    p = s["program"]
    vr = p.vr
    if op == "route":
        vr.vr_route(p.comm, p.logits, p.dtype, case["T"], case["K"], case["E"], p.topk_idx, p.weights, p.flags)
        return {"topk_idx": s["topk_idx"], "weights": s["weights"]}
    if op == "route_backward":
        vr.vr_route_backward(p.comm, p.logits, p.dtype, case["T"], case["K"], case["E"], p.topk_idx, p.weights, p.dweights,
                             p.dlogits, p.flags)
        return s["dlogits"]
    if op == "linear":
        vr.vr_linear(p.comm, p.shape, p.x, p.w, p.out, bias=p.bias, residual=p.residual, group_rows=p.group_rows,
                     workspace=p.workspace, workspace_bytes=p.workspace_bytes)
        return s["out"]
    if op == "linear_backward":
        vr.vr_linear_backward(p.comm, p.shape, p.dout, p.x, p.w, preact=p.preact, dx=p.dx, dw=p.dw, dbias=p.dbias,
                              group_rows=p.group_rows, workspace=p.workspace, workspace_bytes=p.workspace_bytes)
        return {k: s[k] for k in (("dx", "dw", "dbias") if case["bias"] else ("dx", "dw"))}
    vr.vr_moe_layer(p.comm, p.shape, p.x, p.router, p.w_up, p.w_down, p.out, p.topk_idx, p.weights, residual=p.residual,
                    workspace=p.workspace, workspace_bytes=p.workspace_bytes)
    return {"out": s["out"], "topk_idx": s["topk_idx"], "weights": s["weights"]}


# ---- what a pass cannot do without -------------------------------------------------------------
def work(case):
    op, R = case["op"], case["R"]
    esize = 4 if case["dtype"] == "f32" else 2
    if op in ("route", "route_backward"):
        n, tk = R * case["T"] * case["E"], R * case["T"] * case["K"]
        if op == "route":
            return {"bytes": n * esize + tk * 8, "flops": 4 * n}
        return {"bytes": n * esize * (1 if case["renorm"] else 2) + tk * 12, "flops": (1 if case["renorm"] else 6) * n}
    if op == "moe":
        N, E, K, H, I = R * case["T"], case["E"], case["K"], case["H"], case["I"]
        used = E * (1 - (1 - K / E) ** N)  # experts that at least one token chooses, on average
        mats = 3 if case["gated"] else 2
        rows = N * H * (3 if case["residual"] else 2)
        return {"bytes": (used * mats * H * I + E * H + rows) * esize + N * K * 8, "flops": 2 * N * (E * H + K * mats * H * I)}
    G, rows, I, O = case["G"], case["rows"], case["I"], case["O"]
    N = 2 * O if case["gated"] else O
    used = rows - rows // 16 if G > 1 else rows
    w, b = R * min(G, used) * N * I, R * min(G, used) * N if case["bias"] else 0
    if op == "linear":
        return {"bytes": (R * used * (I + O * (2 if case["residual"] else 1)) + w + b) * esize, "flops": 2 * R * used * N * I}
    z = 0 if case["act"] == "none" and not case["gated"] else N
    return {"bytes": (R * used * (O + z + 2 * I) + w + R * G * N * I + b) * esize, "flops": 4 * R * used * N * I}


# ---- the definition in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "route_backward": _exact_route_backward, "linear": _exact_linear,
            "linear_backward": _exact_linear_backward, "moe": _exact_moe}[case["op"]](s, case)


def _softmax64(v):
    m = v.max(-1, keepdim=True).values
    m = torch.nan_to_num(m, neginf=0.0)
    w = (v - m).exp()
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, w / total, torch.zeros_like(w))


def _exact_route(s, case):
    v = s["logits"].double()
    prob = _softmax64(v)
    left, ids, got = v.clone(), [], []
    index = torch.arange(case["E"], device=v.device).expand_as(v)
    for _ in range(case["K"]):  # the largest that is left, the lowest of those that are equal
        best = left.max(-1, keepdim=True).values
        k = torch.where(left == best, index, case["E"]).min(-1, keepdim=True).values
        none = best == -math.inf
        ids.append(torch.where(none, -1, k))
        got.append(torch.where(none, 0.0, prob.gather(-1, k)))
        left.scatter_(-1, k, -math.inf)
    ids, got = torch.cat(ids, -1), torch.cat(got, -1)
    if case["renorm"]:
        total = got.sum(-1, keepdim=True)
        got = torch.where(total > 0, got / total, 0.0)
    return {"topk_idx": ids.to(torch.int32), "weights": got}


def _exact_route_backward(s, case):
    v, idx = s["logits"].double(), s["topk_idx"].long()
    dw, w = s["dweights"].double(), s["weights"].double()
    grad = torch.zeros_like(v)
    have = idx >= 0
    inner = (torch.where(have, dw, 0.0) * w).sum(-1)
    p = None if case["renorm"] else _softmax64(v)
    for k in range(case["K"]):
        at = idx[..., k:k + 1].clamp(min=0)
        g = torch.where(have[..., k:k + 1], dw[..., k:k + 1], 0.0)
        scale = w[..., k:k + 1] if case["renorm"] else p.gather(-1, at)
        grad.scatter_add_(-1, at, torch.where(have[..., k:k + 1], scale * (g - (inner[..., None] if case["renorm"] else 0.0)), 0.0))
    return grad if case["renorm"] else grad - p * inner[..., None]


def _each_group(s, case):
    """(rank, group, first row, past the last) of every group with rows, and of the one group of a dense layer."""
    for r in range(case["R"]):
        at = 0
        counts = [case["rows"]] if s["group_rows"] is None else s["group_rows"][r].tolist()
        for g, n in enumerate(counts):
            yield r, g, at, at + n
            at += n


def _act64(v, name):
    sigma = torch.sigmoid
    normal = torch.distributions.Normal(torch.zeros((), dtype=v.dtype, device=v.device), torch.ones((), dtype=v.dtype, device=v.device))
    if name == "gelu":
        return v * normal.cdf(v), normal.cdf(v) + v * normal.log_prob(v).exp()
    if name == "silu":
        return v * sigma(v), sigma(v) + v * sigma(v) * sigma(-v)
    if name == "relu":
        return v.clamp(min=0), (v > 0).to(v.dtype)
    return v, torch.ones_like(v)


def _exact_linear(s, case):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    O = case["O"]
    for r, g, a, b in _each_group(s, case):
        z = s["x"][r, a:b].double() @ s["w"][r, g].double().T
        if case["bias"]:
            z += s["bias"][r, g].double()
        y = _act64(z[:, :O], case["act"])[0]
        if case["gated"]:
            y = y * z[:, O:]
        if case["residual"]:
            y = y + s["residual"][r, a:b].double()
        out[r, a:b] = y
    return out


def _exact_linear_backward(s, case):
    got = {"dx": torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda"),
           "dw": torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")}
    if case["bias"]:
        got["dbias"] = torch.zeros(s["bias"].shape, dtype=torch.float64, device="cuda")
    O = case["O"]
    for r, g, a, b in _each_group(s, case):
        d = s["dout"][r, a:b].double()
        if s["preact"] is not None:
            z = s["preact"][r, a:b].double()
            y, slope = _act64(z[:, :O], case["act"])
            d = torch.cat([d * z[:, O:] * slope, d * y], 1) if case["gated"] else d * slope
        got["dx"][r, a:b] = d @ s["w"][r, g].double()
        got["dw"][r, g] = d.T @ s["x"][r, a:b].double()
        if case["bias"]:
            got["dbias"][r, g] = d.sum(0)
    return got


def _exact_moe(s, case):
    R, T, K, H, I, E = (case[k] for k in ("R", "T", "K", "H", "I", "E"))
    x = s["x"].reshape(R * T, H).double()
    v = (x[:, None, :] * s["router"].double()[None]).sum(-1)
    chosen = _exact_route({"logits": v}, case)
    idx, weight = chosen["topk_idx"], chosen["weights"]
    out = s["residual"].reshape(R * T, H).double().clone() if case["residual"] else torch.zeros(R * T, H, dtype=torch.float64, device="cuda")
    for e in torch.unique(idx).tolist():
        token, slot = torch.nonzero(idx == e, as_tuple=True)
        z = x[token] @ s["w_up"][e // (E // R), e % (E // R)].double().T
        h = _act64(z[:, :I], case["act"])[0]
        if case["gated"]:
            h = h * z[:, I:]
        out.index_add_(0, token, weight[token, slot][:, None] * (h @ s["w_down"][e // (E // R), e % (E // R)].double().T))
    return {"out": out.reshape(R, T, H), "topk_idx": idx.reshape(R, T, K), "weights": weight.reshape(R, T, K)}
