"""The operators around a recurrent token mixer, as cases that can be timed and
compared: the gated linear recurrence over channels (serving step, prefill,
training with packed sequences), the group norm with its activation over the
mixer's heads (forward and backward), and the linear layer in microscaled
4-bit floating point (quantisation of the activations and the product with
stored weights).

Each case is prepared once (`prepare`), run in its plain torch form or through
the library's entry points (`run`, by the module's name `own`), and computed
from its definition in 64 bits (`exact`).
"""

import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"fp32": F32, "bf16": BF16}
BYTES = {"fp32": 4, "bf16": 2}


def listed():
    return [
        # one decode step of a recurrent layer for a serving batch of 64: launch latency is all
        dict(name="scan step b64", kind="scan_step", batch=64, channels=4096, dtype="bf16", logits=True, lerp=True),
        # prefill of four prompts through one layer of 16 heads of 128 channels, continuing earlier states
        dict(name="scan prefill b4", kind="scan", batch=4, tokens=8192, channels=2048, dtype="bf16", logits=True,
             lerp=True, state=True),
        # one document of a quarter of a million tokens: few channels, parallel over time or not at all; fp32
        dict(name="scan long fp32", kind="scan", batch=1, tokens=262144, channels=640, dtype="fp32", logits=False,
             lerp=False, state=False),
        # a training step on packed documents at 80 heads of 64 channels: forward, then every gradient
        dict(name="scan train packed", kind="scan_train", seqs=48, tokens=32768, channels=5120, dtype="bf16",
             logits=True, lerp=True, state=True),
        # the same step at sizes that divide nothing: a small fp32 model, three sequences of odd length
        dict(name="scan train odd", kind="scan_train", seqs=3, tokens=3063, channels=331, dtype="fp32", logits=False,
             lerp=False, state=True),
        # the norm of one decode step's heads, gated: a few hundred kilobytes, latency
        dict(name="norm decode", kind="norm", rows=64, groups=32, width=128, dtype="bf16", gate=True, act="silu",
             center=False, shared=True, bias=False),
        # heads of 128 normalised and gated in training, one weight shared by all heads
        dict(name="norm train heads", kind="norm_train", rows=32768, groups=16, width=128, dtype="bf16", gate=True,
             act="silu", center=False, shared=True, bias=False),
        # one group as wide as the layer, gated, on a long prefill
        dict(name="norm wide", kind="norm", rows=16384, groups=1, width=5120, dtype="bf16", gate=True, act="silu",
             center=False, shared=False, bias=False),
        # odd width, mean removed, weights and biases of every channel, the activation on the norm itself; fp32
        dict(name="norm train odd", kind="norm_train", rows=4099, groups=7, width=171, dtype="fp32", gate=False,
             act="silu", center=True, shared=False, bias=True),
        # the output projection of a decode step: the weights' bytes are the work
        dict(name="mx linear decode", kind="mx", rows=64, cols=4096, depth=4096),
        # a projection of a long prefill: the matrix units are the work
        dict(name="mx linear prefill", kind="mx", rows=16384, cols=8192, depth=4096),
        # ragged everything: rows and columns that end inside a tile, a depth that is no multiple of the tile's
        dict(name="mx linear odd", kind="mx", rows=1001, cols=1111, depth=2080),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["scan_step", "scan", "scan", "scan_train", "scan_train", "norm", "norm_train", "norm_train",
                       "mx", "mx", "mx"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    gates = dict(logits=rng.random() < 0.6, lerp=rng.random() < 0.5)
    if kind == "scan_step":
        return dict(kind=kind, batch=log(1, 1024), channels=log(8, 8192), dtype=dtype, **gates)
    if kind == "scan":
        channels = log(1, 8192)
        tokens = log(1, min(131072, 160_000_000 // channels))
        batch = log(1, max(1, min(256, 160_000_000 // (channels * tokens))))
        return dict(kind=kind, batch=batch, tokens=tokens, channels=channels, dtype=dtype,
                    state=rng.random() < 0.5, **gates)
    if kind == "scan_train":
        channels = log(1, 8192)
        tokens = log(1, min(65536, (150_000_000 if dtype == "bf16" else 75_000_000) // channels))
        return dict(kind=kind, seqs=log(1, min(256, tokens + 2)), tokens=tokens, channels=channels, dtype=dtype,
                    state=rng.random() < 0.5, **gates)
    if kind in ("norm", "norm_train"):
        width = log(8, 8192)
        groups = log(1, max(1, min(64, 8192 // width)))
        rows = log(1, min(131072, 60_000_000 // (width * groups)))
        gate = rng.random() < 0.6
        return dict(kind=kind, rows=rows, groups=groups, width=width, dtype=dtype, gate=gate,
                    act=rng.choice(["silu", "sigmoid"] if gate else ["none", "silu", "sigmoid"]),
                    center=rng.random() < 0.4, shared=rng.random() < 0.5, bias=rng.random() < 0.4)
    depth = 32 * log(1, 256)
    cols = log(16, 8192)
    rows = log(1, min(16384, 500_000_000_000 // (depth * cols)))
    return dict(kind=kind, rows=rows, cols=cols, depth=depth)


def work(c):
    if c["kind"] == "scan_step":
        n, s = c["batch"] * c["channels"], BYTES[c["dtype"]]
        return {"bytes": n * (3 * s + 8), "flops": 8 * n}
    if c["kind"] == "scan":
        n, s = c["batch"] * c["tokens"] * c["channels"], BYTES[c["dtype"]]
        states = c["batch"] * c["channels"] * 4 * (2 if c["state"] else 1)
        return {"bytes": 3 * n * s + states, "flops": 8 * n}
    if c["kind"] == "scan_train":  # x, gate and dy in; y, dx and dgate out
        n, s = c["tokens"] * c["channels"], BYTES[c["dtype"]]
        states = c["seqs"] * c["channels"] * 4 * (4 if c["state"] else 1)
        return {"bytes": 6 * n * s + states, "flops": 28 * n}
    if c["kind"] in ("norm", "norm_train"):
        n, s = c["rows"] * c["groups"] * c["width"], BYTES[c["dtype"]]
        params = c["width"] * (1 if c["shared"] else c["groups"]) * 4 * (2 if c["bias"] else 1)
        arrays = 3 if c["gate"] else 2
        if c["kind"] == "norm":
            return {"bytes": arrays * n * s + params, "flops": 12 * n}
        return {"bytes": (2 * arrays) * n * s + 2 * params, "flops": 36 * n}
    m, n, k = c["rows"], c["cols"], c["depth"]
    return {"bytes": 2 * m * k + n * k // 2 + n * k // 32 + 2 * m * n, "flops": 2 * m * n * k}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype=F32, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=F32)
    if scale != 1.0 or shift != 0.0:
        x = x.mul_(scale).add_(shift)
    return x.to(dtype)


def _gates(g, shape, dtype, logits):
    """Decays near 1, as trained recurrences have them: exp(-softplus(z)), z ~
    N(-3, 0.5), given as they are or as the logits of the same decays."""
    z = torch.randn(shape, generator=g, device="cuda", dtype=F32).mul_(0.5).sub_(3.0)
    if logits:  # sigmoid(-z) = exp(-softplus(z))
        return z.neg_().to(dtype)
    return torch.nn.functional.softplus(z).neg_().exp_().to(dtype)


def _lengths(c, seed):
    """Packed documents: uneven lengths, a few of them empty."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, c["tokens"] + 1, (c["seqs"] - 1,), generator=g).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([c["tokens"]])]).to(torch.int32)


def prepare(case, seed):
    c, kind = case, case["kind"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(c)}
    if kind == "scan_step":
        shape, dt = (c["batch"], c["channels"]), TYPES[c["dtype"]]
        s.update(x=_normal(g, shape, dt), gate=_gates(g, shape, dt, c["logits"]), h=_normal(g, shape),
                 h_next=torch.empty(shape, device="cuda"), y=torch.empty(shape, device="cuda", dtype=dt))
    elif kind == "scan":
        shape, dt = (c["batch"], c["tokens"], c["channels"]), TYPES[c["dtype"]]
        s.update(x=_normal(g, shape, dt), gate=_gates(g, shape, dt, c["logits"]),
                 h0=_normal(g, (c["batch"], c["channels"])) if c["state"] else None)
    elif kind == "scan_train":
        shape, dt = (c["tokens"], c["channels"]), TYPES[c["dtype"]]
        states = (c["seqs"], c["channels"])
        s.update(x=_normal(g, shape, dt), gate=_gates(g, shape, dt, c["logits"]), dy=_normal(g, shape, dt),
                 cu=_lengths(c, seed).cuda(),
                 h0=_normal(g, states) if c["state"] else None,
                 dh_last=_normal(g, states) if c["state"] else None)
    elif kind in ("norm", "norm_train"):
        shape, dt = (c["rows"], c["groups"], c["width"]), TYPES[c["dtype"]]
        pshape = (c["width"],) if c["shared"] else (c["groups"], c["width"])
        # a mixer's outputs: heads of different size, a little off centre
        size = torch.randn((1, c["groups"], 1), generator=g, device="cuda").mul_(0.7).exp_()
        s.update(x=_normal(g, shape, F32, 1.0, 0.1).mul_(size).to(dt),
                 gate=_normal(g, shape, dt, 1.5) if c["gate"] else None,
                 weight=_normal(g, pshape, F32, 0.2, 1.0),
                 bias=_normal(g, pshape, F32, 0.2) if c["bias"] else None)
        if kind == "norm_train":
            s["dy"] = _normal(g, shape, dt)
    else:
        x = _normal(g, (c["rows"], c["depth"]))
        x[:, :: 64] *= 8.0  # channels of larger size, as activations have them
        w = _normal(g, (c["cols"], c["depth"]), F32, c["depth"] ** -0.5)
        codes, exponents = _mx_codes(w)
        s.update(x=x.to(BF16), w_codes=codes, w_scales=exponents)
    return s


# ---------------------------------------------------------------- run

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    kind = c["kind"]
    if kind == "scan_step":
        a, b = _plain_gates(s["x"], s["gate"], c)
        h = a * s["h"] + b
        return {"y": h.to(TYPES[c["dtype"]]), "h": h}
    if kind == "scan":
        return _plain_scan(s, c)
    if kind == "scan_train":
        return _plain_scan_train(s, c)
    if kind in ("norm", "norm_train"):
        return _plain_norm(s, c)
    return _plain_mx(s)


def _run_own(s, c):
    from quantized_recurrent_state_gdnq_amd import ops

    kind = c["kind"]
    if kind == "scan_step":
        y = ops.gated_scan_step(s["x"], s["gate"], s["h"], logits=c["logits"], lerp=c["lerp"], h_out=s["h_next"],
                                y=s["y"])
        return {"y": y, "h": s["h_next"]}
    if kind == "scan":
        y, h = ops.gated_scan(s["x"], s["gate"], s["h0"], logits=c["logits"], lerp=c["lerp"])
        return {"y": y, "h": h}
    if kind == "scan_train":
        form = dict(logits=c["logits"], lerp=c["lerp"])
        y, h, carry = ops.gated_scan(s["x"], s["gate"], s["h0"], s["cu"], save=True, **form)
        dx, dgate, dh0 = ops.gated_scan_backward(s["dy"], s["x"], s["gate"], carry, s["h0"], s["dh_last"], s["cu"],
                                                 **form)
        out = {"y": y, "h": h, "dx": dx, "dgate": dgate}
        if dh0 is not None:
            out["dh0"] = dh0
        return out
    if kind in ("norm", "norm_train"):
        form = dict(act=c["act"], center=c["center"], eps=1e-5)
        y = ops.group_norm(s["x"], s["weight"], s["bias"], s["gate"], **form)
        if kind == "norm":
            return {"y": y}
        dx, dgate, dweight, dbias = ops.group_norm_backward(s["dy"], s["x"], s["weight"], s["bias"], s["gate"], **form)
        out = {"y": y, "dx": dx, "dweight": dweight}
        if c["gate"]:
            out["dgate"] = dgate
        if c["bias"]:
            out["dbias"] = dbias
        return out
    return {"y": ops.mx_linear(s["x"], s["w_codes"], s["w_scales"])}


# ---------------------------------------------------------------- plain forms

def _plain_gates(x, gate, c):
    gate = gate.float()
    a = torch.sigmoid(gate) if c["logits"] else gate
    if not c["lerp"]:
        return a, x.to(F32, copy=True)  # the callers add the first states to it
    return a, (torch.sigmoid(-gate) if c["logits"] else 1.0 - gate) * x.float()


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension from h = 0, in
    log2(T) doublings: after each, every row spans twice as many steps."""
    d = 1
    while d < a.shape[0]:
        b = torch.cat([b[:d], torch.addcmul(b[d:], a[d:], b[:-d])])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_scan(s, c):
    a, b = _plain_gates(s["x"], s["gate"], c)
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _recurrence(a.transpose(0, 1), b.transpose(0, 1)).transpose(0, 1)
    return {"y": h.to(TYPES[c["dtype"]]).contiguous(), "h": h[:, -1].contiguous()}


def _plain_scan_train(s, c):
    dt, cu = TYPES[c["dtype"]], s["cu"].long()
    x, dy = s["x"].float(), s["dy"].float()
    a, b = _plain_gates(s["x"], s["gate"], c)
    full = cu[1:] > cu[:-1]  # a sequence without tokens has no first or last row
    first, last = cu[:-1][full], cu[1:][full] - 1
    state = torch.zeros((c["seqs"], c["channels"]), device=x.device) if s["h0"] is None else s["h0"]
    b[first] += a[first] * state[full]
    cut = a.clone()
    cut[first] = 0.0
    h = _recurrence(cut, b)
    h_last = state.clone()
    h_last[full] = h[last]
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = state[full]
    # lambda_t = dy_t + a_{t+1} lambda_{t+1}: the same recurrence, from the back
    dh = dy.clone()
    if s["dh_last"] is not None:
        dh[last] += s["dh_last"][full]
    nxt = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    lam = _recurrence(nxt.flip(0), dh.flip(0)).flip(0)
    gate = s["gate"].float()
    keep = torch.sigmoid(-gate) if c["logits"] else 1.0 - gate  # 1 - a
    dx = lam * keep if c["lerp"] else lam
    dgate = lam * (before - x if c["lerp"] else before)
    if c["logits"]:
        dgate = dgate * a * keep
    out = {"y": h.to(dt), "h": h_last, "dx": dx.to(dt), "dgate": dgate.to(dt)}
    if s["h0"] is not None:
        dh0 = s["dh_last"].clone()
        dh0[full] = a[first] * lam[first]
        out["dh0"] = dh0
    return out


def _act(n, act):
    """The activation and its derivative."""
    if act == "none":
        return n, torch.ones_like(n)
    p = torch.sigmoid(n)
    if act == "sigmoid":
        return p, p * (1 - p)
    return n * p, p * (1 + n * (1 - p))


def _plain_norm(s, c):
    dt = TYPES[c["dtype"]]
    x, w = s["x"].float(), s["weight"]
    if c["center"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    hat = x * rstd
    n = hat * w
    if s["bias"] is not None:
        n = n + s["bias"]
    gate = n if s["gate"] is None else s["gate"].float()
    value, slope = _act(gate, c["act"])
    y = value if s["gate"] is None else n * value
    if c["kind"] == "norm":
        return {"y": y.to(dt)}
    dy = s["dy"].float()
    dn = dy * slope if s["gate"] is None else dy * value
    over = (0, 1) if c["shared"] else 0
    dhat = dn * w
    dx = dhat - hat * (dhat * hat).mean(-1, keepdim=True)
    if c["center"]:
        dx = dx - dhat.mean(-1, keepdim=True)
    out = {"y": y.to(dt), "dx": (dx * rstd).to(dt), "dweight": (dn * hat).sum(over)}
    if s["gate"] is not None:
        out["dgate"] = (dy * n * slope).to(dt)
    if s["bias"] is not None:
        out["dbias"] = dn.sum(over)
    return out


def _mx_blocks(x):
    """Values on the 4-bit grid (0, .5, 1, 1.5, 2, 3, 4, 6 with a sign) and the
    power of two of every 32 values: two below the largest's own."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    q = torch.ldexp(b, -e)
    m = q.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign((torch.round(m / step) * step).clamp(max=6.0), q), e


def _mx_codes(x):
    """The stored form: two 4-bit codes a byte, the even column in the low
    nibble, and one exponent byte (bias 127) per 32 values."""
    v, e = _mx_blocks(x)
    m = v.abs()
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), (e + 127).squeeze(-1).to(torch.uint8).contiguous()


def _mx_values(codes, exponents):
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    return torch.ldexp(grid[pair.int()].unflatten(-1, (-1, 32)), exponents.int().unsqueeze(-1) - 127).flatten(-2)


def _plain_mx(s):
    v, e = _mx_blocks(s["x"])
    a = torch.ldexp(v, e).flatten(-2)
    return {"y": (a @ _mx_values(s["w_codes"], s["w_scales"]).t()).to(BF16)}


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    c, s = case, prepare(case, seed)
    wide = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if c["kind"].startswith("scan"):
        a = 1 / (1 + torch.exp(-wide["gate"])) if c["logits"] else wide["gate"]
        keep = 1 / (1 + torch.exp(wide["gate"])) if c["logits"] else 1 - wide["gate"]
        b = keep * wide["x"] if c["lerp"] else wide["x"]
        if c["kind"] == "scan_step":
            h = a * wide["h"] + b
            return {"y": h, "h": h}
        if c["kind"] == "scan":
            h = wide["h0"] if c["state"] else torch.zeros_like(b[:, 0])
            y = torch.empty_like(b)
            for t in range(c["tokens"]):
                h = torch.addcmul(b[:, t], a[:, t], h)
                y[:, t] = h
            return {"y": y, "h": h}
        return _exact_scan_train(wide, c, a, keep, b, s["cu"].tolist())
    if c["kind"].startswith("norm"):
        return _exact_norm(wide, c)
    return _exact_mx(wide, s)


def _exact_scan_train(s, c, a, keep, b, cu):
    zero = torch.zeros(c["channels"], dtype=torch.float64, device=a.device)
    y, lam, before = torch.empty_like(b), torch.empty_like(b), torch.empty_like(b)
    h_last, dh0 = [], []
    for i in range(c["seqs"]):
        h = s["h0"][i] if c["state"] else zero
        for t in range(cu[i], cu[i + 1]):
            before[t] = h
            h = torch.addcmul(b[t], a[t], h)
            y[t] = h
        h_last.append(h)
        m = s["dh_last"][i] if c["state"] else zero
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            m = s["dy"][t] + m
            lam[t] = m
            m = a[t] * m
        dh0.append(m)
    dgate = lam * (before - s["x"] if c["lerp"] else before) * (a * keep if c["logits"] else 1.0)
    out = {"y": y, "h": torch.stack(h_last), "dx": lam * keep if c["lerp"] else lam, "dgate": dgate}
    if c["state"]:
        out["dh0"] = torch.stack(dh0)
    return out


def _exact_norm(s, c):
    x, w = s["x"], s["weight"]
    mu = x.sum(-1, keepdim=True) / c["width"] if c["center"] else 0.0
    sigma = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / c["width"] + 1e-5)
    hat = (x - mu) / sigma
    n = hat * w + (s["bias"] if c["bias"] else 0.0)
    u = s["gate"] if c["gate"] else n
    p = 1 / (1 + torch.exp(-u))
    f = {"none": u, "sigmoid": p, "silu": u * p}[c["act"]]
    df = {"none": torch.ones_like(u), "sigmoid": p * (1 - p), "silu": p + u * p * (1 - p)}[c["act"]]
    out = {"y": n * f if c["gate"] else f}
    if c["kind"] == "norm":
        return out
    dn = s["dy"] * (f if c["gate"] else df)
    axes = [0, 1] if c["shared"] else [0]
    dhat = dn * w
    inner = (dhat * hat).sum(-1, keepdim=True) / c["width"]
    mean = dhat.sum(-1, keepdim=True) / c["width"] if c["center"] else 0.0
    out.update(dx=(dhat - mean - hat * inner) / sigma, dweight=(dn * hat).sum(axes))
    if c["gate"]:
        out["dgate"] = s["dy"] * n * df
    if c["bias"]:
        out["dbias"] = dn.sum(axes)
    return out


def _exact_mx(wide, s):
    """Each block's scale is 2^(floor(log2 max) - 2); a value goes to the
    nearest of the eight magnitudes, half-way ones to the even code."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=s["x"].device)
    middle = (grid[1:] + grid[:-1]) / 2
    b = wide["x"].unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    mantissa, exponent = torch.frexp(torch.where(top > 0, top, 1.0))
    scale = torch.ldexp(torch.ones_like(mantissa), exponent - 3)
    m = (b / scale).abs()
    below = torch.bucketize(m, middle)  # middles under m
    tie_up = (m.unsqueeze(-1) == middle[1::2]).any(-1)  # from an odd code to the even one above
    a = (torch.sign(b) * grid[below + tie_up] * scale).flatten(-2)
    low, high = s["w_codes"].int() & 15, s["w_codes"].int() >> 4
    code = torch.stack([low, high], -1).flatten(-2)
    w = torch.where(code >= 8, -1.0, 1.0) * grid[code % 8]
    w = (w.unflatten(-1, (-1, 32)) * 2.0 ** (s["w_scales"].double().unsqueeze(-1) - 127)).flatten(-2)
    return {"y": a @ w.t().contiguous()}
