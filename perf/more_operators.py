"""The operators of a gated delta-rule layer that is trained, or served with its
state in fp32, as cases that can be timed and compared: the delta rule itself
(serving step, prefill, training with packed sequences), the norm of its
queries and keys with the position rotation (forward and backward), and the
projections in 8-bit integers with a scale for every token and channel.

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
CHUNK = 64  # tokens that the plain delta rule takes at once


def listed():
    return [
        # one sequence's next token through one layer: launch latency is all
        dict(name="delta step b1", kind="delta_step", batch=1, key_heads=16, heads=16, dk=128, dv=128, dtype="bf16",
             log=False),
        # the decode step of a serving batch of 64: the states' bytes are the work
        dict(name="delta step b64", kind="delta_step", batch=64, key_heads=16, heads=32, dk=128, dv=128, dtype="bf16",
             log=False),
        # prefill of four prompts of 8192 tokens, continuing earlier states
        dict(name="delta prefill b4", kind="delta", batch=4, tokens=8192, key_heads=16, heads=16, dk=128, dv=128,
             log=False, state=True),
        # one document of 64 thousand tokens through a layer of few heads: parallel over time or not at all
        dict(name="delta long", kind="delta", batch=1, tokens=65536, key_heads=4, heads=8, dk=128, dv=128, log=True,
             state=False),
        # a training step on packed documents, two value heads to a key head: forward, then every gradient
        dict(name="delta train packed", kind="delta_train", seqs=12, tokens=16384, key_heads=8, heads=16, dk=128,
             dv=128, log=True, state=True),
        # the same step at sizes that divide nothing
        dict(name="delta train odd", kind="delta_train", seqs=3, tokens=1003, key_heads=2, heads=6, dk=72, dv=104,
             log=False, state=True),
        # the queries and keys of one decode step, out of the fused projection's rows: latency
        dict(name="qk norm decode", kind="qk", rows=64, q_heads=16, k_heads=16, dim=128, rotary=32, dtype="bf16",
             norm="rms", weights=True, interleaved=False, fused=True, far=1 << 17),
        # training: every head normalised with its weight and rotated, then the gradients
        dict(name="qk norm train", kind="qk_train", rows=32768, q_heads=32, k_heads=8, dim=128, rotary=128,
             dtype="bf16", norm="rms", weights=True, interleaved=False, fused=True, far=32768),
        # a small fp32 model with odd heads, pairs side by side, positions far out
        dict(name="qk norm train odd", kind="qk_train", rows=4099, q_heads=7, k_heads=3, dim=90, rotary=38,
             dtype="fp32", norm="l2", weights=False, interleaved=True, fused=False, far=1 << 22),
        # the output projection of a decode step: the weights' bytes are the work
        dict(name="int8 linear decode", kind="int8", rows=64, cols=4096, depth=4096, dtype="bf16", bias=False),
        # a projection of a long prefill: the matrix units are the work
        dict(name="int8 linear prefill", kind="int8", rows=16384, cols=8192, depth=4096, dtype="bf16", bias=False),
        # rows quantized once for two projections, at sizes that end inside every tile; fp32 in and out
        dict(name="int8 two projections odd", kind="int8_two", rows=1001, cols=1111, depth=2064, dtype="fp32",
             bias=True),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["delta_step", "delta", "delta", "delta_train", "delta_train", "delta_train", "qk", "qk_train",
                       "qk_train", "int8", "int8", "int8_two"])
    if kind.startswith("delta"):
        dk = rng.choice([64, 128, 128, 8 * rng.randint(1, 16)])
        dv = rng.choice([64, 128, 128, 8 * rng.randint(1, 32)])
        key_heads = log(1, 16)
        heads = key_heads * rng.choice([1, 1, 2, 3])
        c = dict(kind=kind, key_heads=key_heads, heads=heads, dk=dk, dv=dv, log=rng.random() < 0.5)
        if kind == "delta_step":
            return dict(c, batch=log(1, max(1, 33_000_000 // (heads * dk * dv))), dtype=rng.choice(["bf16", "bf16", "fp32"]))
        most = (520_000_000 if kind == "delta" else 220_000_000) // (heads * max(dk * dv // 128, 64))
        tokens = log(1, min(32768, most))
        c.update(tokens=tokens, state=tokens < 512 or rng.random() < 0.5)
        if kind == "delta":
            return dict(c, batch=log(1, max(1, min(64, most // tokens))))
        return dict(c, seqs=log(1, min(64, tokens + 2)))
    if kind.startswith("qk"):
        dim = rng.choice([64, 128, 128, rng.randint(4, 256)])
        q_heads = log(1, 64)
        k_heads = rng.choice([q_heads, max(1, q_heads // rng.choice([2, 4, 8]))])
        rows = log(1, min(65536, 160_000_000 // (dim * (q_heads + k_heads))))
        rotary = rng.choice([0, dim // 2 * 2, 2 * rng.randint(1, dim // 2)])
        return dict(kind=kind, rows=rows, q_heads=q_heads, k_heads=k_heads, dim=dim, rotary=rotary,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), norm=rng.choice(["rms", "rms", "l2"]),
                    weights=rng.random() < 0.6, interleaved=rng.random() < 0.3, fused=rng.random() < 0.5,
                    far=log(1, 1 << 22))
    depth = 16 * log(1, 768)
    cols = log(16, 8192)
    rows = log(1, min(16384, (500_000_000_000 if kind == "int8" else 100_000_000_000) // (depth * cols)))
    return dict(kind=kind, rows=rows, cols=cols, depth=depth, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                bias=rng.random() < 0.4)


def work(c):
    kind = c["kind"]
    if kind.startswith("delta"):
        g, h, dk, dv = c["key_heads"], c["heads"], c["dk"], c["dv"]
        one = dk * dv * h  # a token's, or a state's
        if kind == "delta_step":
            n, s = c["batch"], BYTES[c["dtype"]]
            return {"bytes": n * ((2 * g * dk + 2 * h * dv) * s + 8 * h + 8 * one), "flops": 6 * n * one}
        n = c["tokens"] * c.get("batch", 1)
        states = 4 * one * c.get("batch", c.get("seqs"))
        if kind == "delta":
            return {"bytes": n * (4 * g * dk + 4 * h * dv + 8 * h) + states * (2 if c["state"] else 1),
                    "flops": 6 * n * one}
        return {"bytes": n * (8 * g * dk + 8 * h * dv + 16 * h) + states * (4 if c["state"] else 1),
                "flops": 20 * n * one}
    if kind.startswith("qk"):
        n, s = c["rows"] * (c["q_heads"] + c["k_heads"]) * c["dim"], BYTES[c["dtype"]]
        params = 8 * c["dim"] if c["weights"] else 0
        pos = (8 * c["rows"] + 2 * c["rotary"]) if c["rotary"] else 0
        if kind == "qk":
            return {"bytes": 2 * n * s + params + pos, "flops": 8 * n}
        return {"bytes": 4 * n * s + 2 * params + pos, "flops": 24 * n}
    m, n, k, s = c["rows"], c["cols"], c["depth"], BYTES[c["dtype"]]
    times = 2 if kind == "int8_two" else 1
    return {"bytes": s * m * k + times * (n * k + 4 * n + s * m * n + (4 * n if c["bias"] else 0))
            + (m * k + 4 * m if times == 2 else 0),
            "flops": times * 2 * m * n * k}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype=F32, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=F32)
    if scale != 1.0 or shift != 0.0:
        x = x.mul_(scale).add_(shift)
    return x.to(dtype)


def _keys(g, lead, heads, dim, dtype):
    """Unit vectors that lean towards one direction of their head, as trained
    keys do."""
    x = _normal(g, lead + (heads, dim))
    x = x + 0.5 * _normal(g, (heads, dim))
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _lengths(c, seed):
    """Packed documents: uneven lengths, a few of them empty."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, c["tokens"] + 1, (c["seqs"] - 1,), generator=g).sort().values.tolist()
    ends = cuts + [c["tokens"]]
    return [b - a for a, b in zip([0] + cuts, ends)]


def prepare(case, seed):
    c, kind = case, case["kind"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(c)}
    if kind.startswith("delta"):
        dt = TYPES[c.get("dtype", "bf16")]
        lead = {"delta_step": (c.get("batch"),), "delta": (c.get("batch"), c.get("tokens"))}.get(kind, (c.get("tokens"),))
        states = (c.get("batch", c.get("seqs")), c["heads"], c["dv"], c["dk"])
        decay = -torch.nn.functional.softplus(_normal(g, lead + (c["heads"],), F32, 0.5, -3.0))
        s.update(q=_keys(g, lead, c["key_heads"], c["dk"], dt), k=_keys(g, lead, c["key_heads"], c["dk"], dt),
                 v=_normal(g, lead + (c["heads"], c["dv"]), dt), alpha=decay if c["log"] else decay.exp(),
                 beta=torch.sigmoid(_normal(g, lead + (c["heads"],))))
        if kind == "delta_step":
            s.update(h=_normal(g, states, F32, 0.5), h_next=torch.empty(states, device="cuda"),
                     o=torch.empty(lead + (c["heads"], c["dv"]), device="cuda", dtype=dt))
            return s
        s["h0"] = _normal(g, states, F32, 0.5) if c["state"] else None
        if kind == "delta_train":
            s["lengths"] = _lengths(c, seed)
            s["cu"] = torch.tensor([0] + s["lengths"], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
            s["do"] = _normal(g, lead + (c["heads"], c["dv"]), BF16)
            s["dh_last"] = _normal(g, states, F32, 0.5) if c["state"] else None
    elif kind.startswith("qk"):
        dt, n, d = TYPES[c["dtype"]], c["rows"], c["dim"]
        qw, kw = c["q_heads"] * d, c["k_heads"] * d
        if c["fused"]:  # views of the rows of one projection, which go on with the values
            rows = _normal(g, (n, (qw + 2 * kw + 7) // 8 * 8), dt)
            q, k = rows[:, :qw].unflatten(-1, (-1, d)), rows[:, qw:qw + kw].unflatten(-1, (-1, d))
        else:
            q, k = _normal(g, (n, c["q_heads"], d), dt), _normal(g, (n, c["k_heads"], d), dt)
        s.update(q=q, k=k, q_weight=None, k_weight=None, positions=None, inv_freq=None)
        if c["weights"]:
            s.update(q_weight=_normal(g, (d,), F32, 0.2, 1.0), k_weight=_normal(g, (d,), F32, 0.2, 1.0))
        if c["rotary"]:
            s["positions"] = torch.randint(0, c["far"], (n,), generator=g, device="cuda")
            pairs = torch.arange(0, c["rotary"], 2, dtype=torch.float64, device="cuda")
            s["inv_freq"] = (10000.0 ** (-pairs / c["rotary"])).float()
        if kind == "qk_train":
            s.update(dq_out=_normal(g, (n, c["q_heads"], d), dt), dk_out=_normal(g, (n, c["k_heads"], d), dt))
    else:
        x = _normal(g, (c["rows"], c["depth"]))
        x[:, ::64] *= 8.0  # channels of larger size, as activations have them
        s["x"] = x.to(TYPES[c["dtype"]])
        for name in ("w", "u") if kind == "int8_two" else ("w",):
            codes, scales = _codes(_normal(g, (c["cols"], c["depth"]), F32, c["depth"] ** -0.5))
            s.update({name + "_codes": codes, name + "_scales": scales,
                      name + "_bias": _normal(g, (c["cols"],)) if c["bias"] else None})
    return s


# ---------------------------------------------------------------- run

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    kind = c["kind"]
    if kind == "delta_step":
        return _plain_step(s, c)
    if kind.startswith("delta"):
        return _plain_delta(s, c)
    if kind.startswith("qk"):
        return _plain_qk(s, c)
    codes, scales = _codes(s["x"])
    out = {"y": _plain_product(codes, scales, s, "w", TYPES[c["dtype"]])}
    if kind == "int8_two":
        out.update(codes=codes, scales=scales, y2=_plain_product(codes, scales, s, "u", TYPES[c["dtype"]]))
    return out


def _run_own(s, c):
    from quantized_recurrent_state_gdnq_amd import ops

    kind = c["kind"]
    if kind == "delta_step":
        o = ops.delta_rule_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["h"], log_decay=c["log"],
                                h_out=s["h_next"], o=s["o"])
        return {"o": o, "h": s["h_next"]}
    if kind == "delta":
        o, h = ops.delta_rule(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["h0"], log_decay=c["log"])
        return {"o": o, "h": h}
    if kind == "delta_train":
        args = s["q"], s["k"], s["v"], s["alpha"], s["beta"]
        o, h, carry = ops.delta_rule(*args, s["h0"], s["cu"], log_decay=c["log"], save=True)
        dq, dk, dv, dalpha, dbeta, dh0 = ops.delta_rule_backward(s["do"], *args, carry, s["h0"], s["dh_last"], s["cu"],
                                                                 log_decay=c["log"])
        out = {"o": o, "h": h, "dq": dq, "dk": dk, "dv": dv, "dalpha": dalpha, "dbeta": dbeta}
        if dh0 is not None:
            out["dh0"] = dh0
        return out
    if kind.startswith("qk"):
        args = s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"]
        form = dict(norm=c["norm"], eps=1e-6, interleaved=c["interleaved"])
        q, k = ops.qk_norm(*args, **form)
        if kind == "qk":
            return {"q": q, "k": k}
        dq, dk, dq_weight, dk_weight = ops.qk_norm_backward(s["dq_out"], s["dk_out"], *args, **form)
        out = {"q": q, "k": k, "dq": dq, "dk": dk}
        if c["weights"]:
            out.update(dq_weight=dq_weight, dk_weight=dk_weight)
        return out
    if kind == "int8":
        return {"y": ops.int8_linear(s["x"], s["w_codes"], s["w_scales"], s["w_bias"])}
    codes, scales = ops.int8_quantize(s["x"])
    form = dict(out_dtype=TYPES[c["dtype"]])
    return {"y": ops.int8_matmul(codes, scales, s["w_codes"], s["w_scales"], s["w_bias"], **form),
            "codes": codes, "scales": scales,
            "y2": ops.int8_matmul(codes, scales, s["u_codes"], s["u_scales"], s["u_bias"], **form)}


# ---------------------------------------------------------------- plain forms

def _plain_step(s, c):
    share = c["heads"] // c["key_heads"]
    q, k = (s[n].float().repeat_interleave(share, 1).unsqueeze(-2) for n in ("q", "k"))
    a = (s["alpha"].exp() if c["log"] else s["alpha"])[..., None, None]
    h = a * s["h"]
    u = s["beta"].unsqueeze(-1) * (s["v"].float() - (h * k).sum(-1))
    h = h + u.unsqueeze(-1) * k
    return {"o": (h * q).sum(-1).to(TYPES[c["dtype"]]), "h": h}


def _inverse(a):
    """(I + a)^-1 of strictly lower triangles a [.., 64, 64], by blocks: the
    lower left block of the inverse of two blocks is -n2 a21 n1."""
    n = torch.eye(CHUNK, device=a.device).expand_as(a).clone()
    size = 1
    while size < CHUNK:
        pairs = n.unflatten(-1, (-1, 2, size)).unflatten(-4, (-1, 2, size))  # [.., pair, 2, size, pair, 2, size]
        diagonal = lambda x, i, j: torch.stack([x[..., p, i, :, p, j, :] for p in range(CHUNK // (2 * size))], -3)  # noqa: E731
        block = a.unflatten(-1, (-1, 2, size)).unflatten(-4, (-1, 2, size))
        low = -(diagonal(pairs, 1, 1) @ diagonal(block, 1, 0) @ diagonal(pairs, 0, 0))
        for p in range(CHUNK // (2 * size)):
            at = 2 * size * p
            n[..., at + size:at + 2 * size, at:at + size] = low[..., p, :, :]
        size *= 2
    return n


def _spans(s, c):
    """Where the chunks of every stream lie in the flat tokens: (start, end,
    first of its sequence, last, sequence).  Sequences of equal length are
    streams side by side, packed ones follow each other in one stream."""
    if c["kind"] == "delta":
        t = c["tokens"]
        return [[(b * t + i, min(i + CHUNK, t) + b * t, i == 0, i + CHUNK >= t, b) for i in range(0, t, CHUNK)]
                for b in range(c["batch"])]
    at, stream = 0, []
    for b, n in enumerate(s["lengths"]):
        stream += [(at + i, at + min(i + CHUNK, n), i == 0, i + CHUNK >= n, b) for i in range(0, n, CHUNK)]
        at += n
    return [stream]


def _plain_delta(s, c):
    heads, dk, dv, share = c["heads"], c["dk"], c["dv"], c["heads"] // c["key_heads"]
    spans = _spans(s, c)
    device = s["q"].device
    start, end = (torch.tensor([[p[i] for p in stream] for stream in spans], device=device) for i in (0, 1))
    rows = start.unsqueeze(-1) + torch.arange(CHUNK, device=device)
    here = rows < end.unsqueeze(-1)  # [streams, chunks, 64]
    rows = rows.clamp(max=s["v"].numel() // (heads * dv) - 1)

    def chunks(x, width=None):  # -> [streams, chunks, heads, 64(, width)], zero behind a sequence's end
        x = x.reshape(-1, x.shape[-1] if width is None else x.shape[-2], *(() if width is None else (width,)))
        x = x[rows].float() * (here[..., None] if width is None else here[..., None, None])
        x = x.transpose(2, 3)
        return x if x.shape[2] == heads else x.repeat_interleave(share, 2)

    def flat(x):  # back, in fp32
        x = x.transpose(2, 3)
        out = torch.empty((s["v"].numel() // (heads * dv),) + x.shape[3:], device=device)
        out[rows[here]] = x[here]
        return out

    q, k, v, beta = chunks(s["q"], dk), chunks(s["k"], dk), chunks(s["v"], dv), chunks(s["beta"])
    logs = s["alpha"].double() if c["log"] else s["alpha"].double().log()
    g = (logs.reshape(-1, heads)[rows] * here[..., None]).transpose(2, 3).cumsum(-1)
    ratio = (g.unsqueeze(-1) - g.unsqueeze(-2)).tril().exp().float().tril()
    gamma, tail, whole = g.exp().float().unsqueeze(-1), (g[..., -1:] - g).exp().float().unsqueeze(-1), g[..., -1].exp().float()
    beta = beta.unsqueeze(-1)
    kt = k.transpose(-1, -2)
    a = (ratio * (k @ kt)).tril(-1)
    m = ratio * (q @ kt)
    inverse = _inverse(a * beta.transpose(-1, -2))

    states = torch.zeros((len(s["lengths"]) if "lengths" in s else c["batch"], heads, dv, dk), device=device)
    if s["h0"] is not None:
        states += s["h0"]
    steps = list(zip(*spans))  # the streams' chunks side by side
    tk = tail * k
    before, w = [], []
    for i, at in enumerate(steps):
        seqs = [p[4] for p in at]
        h = states[seqs]
        x = v[:, i] - gamma[:, i] * (k[:, i] @ h.transpose(-1, -2))
        w.append(inverse[:, i] @ x)
        before.append(h)
        states[seqs] = whole[:, i, :, None, None] * h + (beta[:, i] * w[-1]).transpose(-1, -2) @ tk[:, i]
    before, w = torch.stack(before, 1), torch.stack(w, 1)
    u = beta * w
    o = flat(gamma * (q @ before.transpose(-1, -2)) + m @ u).to(BF16)
    if c["kind"] == "delta":
        return {"o": o.view(s["v"].shape), "h": states}

    do = chunks(s["do"], dv)
    back = _inverse(beta * a).transpose(-1, -2).contiguous()
    inner = m.transpose(-1, -2) @ do
    dstates = torch.zeros_like(states)
    if s["dh_last"] is not None:
        dstates += s["dh_last"]
    own_part = do.transpose(-1, -2) @ (gamma * q)
    gk = gamma * k
    after, z = [], []
    for i in reversed(range(len(steps))):
        seqs = [p[4] for p in steps[i]]
        dh = dstates[seqs]
        z.append(back[:, i] @ (inner[:, i] + tail[:, i] * (k[:, i] @ dh.transpose(-1, -2))))
        after.append(dh)
        dstates[seqs] = (whole[:, i, :, None, None] * dh + own_part[:, i]
                         - (beta[:, i] * z[-1]).transpose(-1, -2) @ gk[:, i])
    after, z = torch.stack(after[::-1], 1), torch.stack(z[::-1], 1)
    dx = beta * z
    dm = ratio * (do @ u.transpose(-1, -2))
    da = -ratio * (dx @ u.transpose(-1, -2)).tril(-1)
    dq = gamma * (do @ before) + dm @ k
    ends = tail * (u @ after)
    plus = da @ k - gamma * (dx @ before)
    minus = dm.transpose(-1, -2) @ q + da.transpose(-1, -2) @ k + ends
    # d log alpha_t: all that passes from before token t to it or behind it
    pairs = (dm * (q @ kt) + da * (k @ kt)).flip(-2).cumsum(-2).flip(-2).tril(-1).sum(-1)
    entering = (q * gamma * (do @ before) - k * gamma * (dx @ before)).sum(-1).flip(-1).cumsum(-1).flip(-1)
    leaving = (k * ends).sum(-1)
    leaving = leaving.cumsum(-1) - leaving
    dalpha = flat(pairs + entering + leaving + (whole * (before * after).sum((-1, -2))).unsqueeze(-1))
    if not c["log"]:
        dalpha = dalpha / s["alpha"]
    shared = lambda x: flat(x).unflatten(1, (-1, share)).sum(2).to(BF16)  # noqa: E731
    out = {"o": o, "h": states, "dq": shared(dq), "dk": shared(plus + minus), "dv": flat(dx).to(BF16),
           "dalpha": dalpha, "dbeta": flat((w * z).sum(-1))}
    if s["h0"] is not None:
        out["dh0"] = dstates
    return out


def _angles(s):
    """Angles in 64 bits: 32 lose those of far positions."""
    angle = s["positions"].double().unsqueeze(-1) * s["inv_freq"].double()
    return angle.cos().float().unsqueeze(-2), angle.sin().float().unsqueeze(-2)  # [rows, 1, pairs]


def _rotate(x, cos, sin, c):
    """The first `rotary` columns turned in pairs: (i, i + half), or (2i, 2i + 1)."""
    r = c["rotary"]
    pairs = x[..., :r].unflatten(-1, (-1, 2) if c["interleaved"] else (2, -1))
    dim = -1 if c["interleaved"] else -2
    a, b = pairs.unbind(dim)
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim).flatten(-2), x[..., r:]], -1)


def _plain_qk(s, c):
    dt = TYPES[c["dtype"]]
    turned = _angles(s) if c["rotary"] else None
    out = {}
    for n in ("q", "k"):
        x, weight = s[n].float(), s[n + "_weight"]
        size = (x * x).sum(-1, keepdim=True)
        rstd = torch.rsqrt((size / c["dim"] if c["norm"] == "rms" else size) + 1e-6)
        hat = x * rstd
        y = hat if weight is None else hat * weight
        out[n] = (_rotate(y, *turned, c) if turned else y).to(dt)
        if c["kind"] == "qk_train":
            dy = s["d" + n + "_out"].float()
            if turned:
                dy = _rotate(dy, turned[0], -turned[1], c)
            if weight is not None:
                out["d" + n + "_weight"] = (dy * hat).sum((0, 1))
                dy = dy * weight
            inner = (dy * hat).sum(-1, keepdim=True)
            out["d" + n] = ((dy - hat * (inner / c["dim"] if c["norm"] == "rms" else inner)) * rstd).to(dt)
    return out


def _codes(x):
    """Rows in 8 bits: the scale is a 127th of the largest value, a code the
    nearest whole number to value / scale, half-way ones to the even one."""
    x = x.float()
    scales = x.abs().amax(-1) / torch.full((), 127.0, device=x.device)  # by a number it would be a product with 1 / 127
    codes = torch.round(x / torch.where(scales > 0, scales, torch.ones_like(scales)).unsqueeze(-1))
    return codes.clamp(-127, 127).to(torch.int8), scales


def _plain_product(codes, scales, s, name, dt):
    y = codes.float() @ s[name + "_codes"].float().t()
    y = y * scales.unsqueeze(-1) * s[name + "_scales"]
    return (y if s[name + "_bias"] is None else y + s[name + "_bias"]).to(dt)


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    c, s = case, prepare(case, seed)
    wide = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if c["kind"].startswith("delta"):
        share = c["heads"] // c["key_heads"]
        head = -2
        for n in ("q", "k"):
            wide[n] = wide[n].repeat_interleave(share, head)
        if c["log"]:
            wide["alpha"] = torch.exp(wide["alpha"])
        if c["kind"] == "delta_step":
            h = _token(wide, (), wide["h"])[0]
            return {"o": (h * wide["q"].unsqueeze(-2)).sum(-1), "h": h}
        if c["kind"] == "delta":
            h = wide["h0"] if c["state"] else wide["q"].new_zeros((c["batch"], c["heads"], c["dv"], c["dk"]))
            o = torch.empty_like(wide["v"])
            for t in range(c["tokens"]):
                h = _token(wide, (slice(None), t), h)[0]
                o[:, t] = (h * wide["q"][:, t].unsqueeze(-2)).sum(-1)
            return {"o": o, "h": h}
        return _exact_delta_train(wide, c, s)
    if c["kind"].startswith("qk"):
        return _exact_qk(wide, c)
    return _exact_int8(wide, s, c)


def _token(s, at, h):
    """One token of the recurrence: the state after it, and the error that it
    writes (the value without what the decayed state says of the key)."""
    k = s["k"][at].unsqueeze(-2)
    h = s["alpha"][at][..., None, None] * h
    w = s["v"][at] - (h * k).sum(-1)
    return h + (s["beta"][at].unsqueeze(-1) * w).unsqueeze(-1) * k, w


def _exact_delta_train(s, c, inputs):
    piece = 256  # states are kept for so many tokens at a time, and formed again for the next
    out = {n: torch.zeros_like(s[m]) for n, m in
           (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dalpha", "alpha"), ("dbeta", "beta"))}
    zero = s["q"].new_zeros((c["heads"], c["dv"], c["dk"]))
    h_last, dh0, at = [], [], 0
    for b, n in enumerate(inputs["lengths"]):
        h, marks = (s["h0"][b] if c["state"] else zero), []
        for t in range(at, at + n):
            if (t - at) % piece == 0:
                marks.append(h)
            h = _token(s, t, h)[0]
        h_last.append(h)
        dh = s["dh_last"][b] if c["state"] else zero
        for first in reversed(range(at, at + n, piece)):
            last = min(first + piece, at + n)
            states, errors = [marks[(first - at) // piece]], []
            for t in range(first, last):
                h, w = _token(s, t, states[-1])
                states.append(h)
                errors.append(w)
            for t in reversed(range(first, last)):
                before, after, w = states[t - first], states[t - first + 1], errors[t - first]
                q, k, a, bt = s["q"][t].unsqueeze(-2), s["k"][t].unsqueeze(-2), s["alpha"][t], s["beta"][t].unsqueeze(-1)
                do = s["do"][t].unsqueeze(-1)
                out["o"][t] = (after * q).sum(-1)
                out["dq"][t] = (after * do).sum(-2)
                dh = dh + do * q
                du = (dh * k).sum(-1)
                dw = bt * du
                out["dbeta"][t] = (du * w).sum(-1)
                out["dv"][t] = dw
                out["dalpha"][t] = ((dh - dw.unsqueeze(-1) * k) * before).sum((-1, -2))
                out["dk"][t] = (dh * (bt * w).unsqueeze(-1)).sum(-2) - a.unsqueeze(-1) * (before * dw.unsqueeze(-1)).sum(-2)
                dh = a[..., None, None] * (dh - dw.unsqueeze(-1) * k)
        dh0.append(dh)
        at += n
    for n in ("dq", "dk"):
        out[n] = out[n].unflatten(1, (c["key_heads"], -1)).sum(2)
    if c["log"]:
        out["dalpha"] = out["dalpha"] * s["alpha"]
    out["h"] = torch.stack(h_last)
    if c["state"]:
        out["dh0"] = torch.stack(dh0)
    return {n: out[n] for n in ("o", "h", "dq", "dk", "dv", "dalpha", "dbeta", "dh0") if n in out}


def _exact_qk(s, c):
    """The rotation as a product of complex numbers."""
    d, r = c["dim"], c["rotary"]
    turn = None
    if r:
        turn = torch.exp(1j * (s["positions"].double()[:, None] * s["inv_freq"][None, :]))[:, None, :]

    def rotated(x, turn):
        if turn is None:
            return x
        head = x[..., :r]
        re, im = (head[..., 0::2], head[..., 1::2]) if c["interleaved"] else (head[..., :r // 2], head[..., r // 2:])
        pair = torch.complex(re.contiguous(), im.contiguous()) * turn
        head = torch.view_as_real(pair).flatten(-2) if c["interleaved"] else torch.cat([pair.real, pair.imag], -1)
        return torch.cat([head, x[..., r:]], -1)

    out = {}
    for n in ("q", "k"):
        x = s[n]
        w = s[n + "_weight"] if c["weights"] else torch.ones(d, dtype=torch.float64, device=x.device)
        size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / (d if c["norm"] == "rms" else 1) + 1e-6)
        out[n] = rotated(x / size * w, turn)
        if c["kind"] == "qk_train":
            dy = rotated(s["d" + n + "_out"], None if turn is None else turn.conj())
            # d(x / size) = dx / size - x (x . dx) / size^3 (over the width for the mean)
            out["d" + n] = dy * w / size - x * (x * dy * w).sum(-1, keepdim=True) / (d if c["norm"] == "rms" else 1) / size ** 3
            if c["weights"]:
                out["d" + n + "_weight"] = (dy * x / size).sum((0, 1))
    return out


def _exact_int8(wide, s, c):
    """The codes are settled in 32 bits, as the codec is defined; the product
    is one of whole numbers, exact in 64 bits."""
    top = s["x"].float().abs().max(-1).values
    scale = top / torch.tensor(127.0, device=top.device)
    q = s["x"].float() / scale.clamp_min(torch.finfo(F32).tiny)[:, None]
    low = torch.floor(q)
    rest = q - low
    codes = (low + ((rest > 0.5) | ((rest == 0.5) & (low % 2 != 0))).float()).clamp(-127, 127).double()

    def product(n):
        y = (codes @ s[n + "_codes"].double().t().contiguous()) * (scale.double()[:, None] * wide[n + "_scales"][None])
        return y + wide[n + "_bias"] if c["bias"] else y

    out = {"y": product("w")}
    if c["kind"] == "int8_two":
        out.update(codes=None, scales=top.double() / 127, y2=product("u"))
    return out
