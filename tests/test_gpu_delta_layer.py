"""A mixer layer as its operators are used together: an 8-bit projection to
queries, keys and values in one row, the norm and rotation of the former, the
delta rule with its state in fp32, the gated norm of its heads and an 8-bit
projection back, for a prefill, the decode steps that continue it, a captured
decode step and a training step."""

import pytest
import torch

from gpu_util import DEV
from quantized_recurrent_state_gdnq_amd import ops
from test_gpu_delta_rule import FWD, near, reference

pytestmark = pytest.mark.gpu

G, H, DK, DV, ROT, C = 2, 4, 64, 96, 32, 160
KEYS, COLS = G * DK, 2 * G * DK + H * DV
BF16 = torch.bfloat16


def weights(seed=3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    w_in, w_out = ops.int8_quantize(n(COLS, C) / 8), ops.int8_quantize(n(C, H * DV) / 16)
    freq = (10000.0 ** (-torch.arange(ROT // 2) / (ROT // 2))).to(DEV)
    return dict(w_in=w_in, w_out=w_out, freq=freq, qw=n(DK) * 0.1 + 1, kw=n(DK) * 0.1 + 1, nw=n(DV) * 0.1 + 1)


def inputs(B, T, seed=4):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return (n(B, T, C).to(BF16).to(DEV), n(B, T, H, DV).to(BF16).to(DEV),
            (-torch.nn.functional.softplus(n(B, T, H) - 2)).to(DEV), torch.sigmoid(n(B, T, H)).to(DEV))


def heads(rows, w, positions):
    """q and k of the projected rows [..,COLS], which stay where they are, and v."""
    q, k, v = rows.split([KEYS, KEYS, H * DV], -1)
    q, k = ops.qk_norm(q.unflatten(-1, (G, DK)), k.unflatten(-1, (G, DK)), w["qw"], w["kw"], positions, w["freq"], norm="l2")
    return q, k, v.unflatten(-1, (H, DV)).contiguous()


def back(o, z, w):
    n = ops.group_norm(o, w["nw"], gate=z, act="silu")
    return ops.int8_linear(n.flatten(-2), *w["w_out"])


def layer(x, z, alpha, beta, h, w, first=0):
    B, T = x.shape[:2]
    rows = ops.int8_linear(x, *w["w_in"])
    positions = torch.arange(first, first + T, device=DEV).expand(B, T).contiguous()
    q, k, v = heads(rows, w, positions)
    o, h = ops.delta_rule(q, k, v, alpha, beta, h, log_decay=True)
    return back(o, z, w), h, (rows, q, k, v, o)


def step(x, z, alpha, beta, h, positions, w):
    q, k, v = heads(ops.int8_linear(x, *w["w_in"]), w, positions)
    return back(ops.delta_rule_step(q, k, v, alpha, beta, h, log_decay=True), z, w)


def test_prefill():
    """Every stage against its definition on what the stage before gave."""
    B, T = 2, 150
    w, (x, z, alpha, beta) = weights(), inputs(B, T)
    y, h, (rows, q, k, v, o) = layer(x, z, alpha, beta, None, w)

    def product(a, b):  # the integers' sums are exact in 64 bits also where they cancel; the scales come after
        (ca, sa), (cb, sb) = a, b
        return (ca.double() @ cb.double().T) * sa.double()[..., None] * sb.double()

    want = product(ops.int8_quantize(x), w["w_in"])
    # exact sums, two fp32 products and a rounding to bf16
    assert ((rows.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + 1e-30).all()
    angle = torch.arange(T, device=DEV).double()[:, None] * w["freq"].double()
    for got, at, weight in ((q, 0, "qw"), (k, KEYS, "kw")):
        n = rows[..., at:at + KEYS].unflatten(-1, (G, DK)).double()
        n = n / torch.sqrt((n * n).sum(-1, keepdim=True) + 1e-6) * w[weight].double()
        a, b, c, s = n[..., :ROT // 2], n[..., ROT // 2:ROT], torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        n = torch.cat([a * c - b * s, a * s + b * c, n[..., ROT:]], -1)
        # 23 u of the pair's magnitudes (at most 1.5 in a row of length about 1) before the rounding
        assert ((got.double() - n).abs() <= 2.0 ** -8 * n.abs() + 23 * 2.0 ** -24 * 1.5).all()
    d = dict(q=q, k=k, v=v, alpha=alpha, beta=beta, h0=None)
    ref = reference(d, [(0, T), (T, 2 * T)], log=True)
    near(o, ref["o"], FWD, "o")
    near(h, ref["h"], FWD, "h")
    n = ops.group_norm(o, w["nw"], gate=z, act="silu")
    want = product(ops.int8_quantize(n.flatten(-2)), w["w_out"])
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + 1e-30).all()


def test_prefill_then_decode():
    B, T, steps = 3, 130, 5
    w, (x, z, alpha, beta) = weights(), inputs(B, T + steps)
    cut = lambda i, j: [t[:, i:j].contiguous() for t in (x, z, alpha, beta)]  # noqa: E731
    whole, last, _ = layer(x, z, alpha, beta, None, w)
    y, h, _ = layer(*cut(0, T), None, w)
    outs = [y]
    for t in range(T, T + steps):
        at = torch.full((B,), t, device=DEV)
        outs.append(step(*(v.squeeze(1) for v in cut(t, t + 1)), h, at, w)[:, None])
    # the projections and norms of a token are the same numbers in both, bit for bit; the states differ by the chunked
    # form's parts
    assert float((h - last).norm() / last.norm()) < FWD
    out = torch.cat(outs, 1).double()
    # an output that rounds to bf16 the other way, and from there to another code: one code in a few hundred, of at most
    # 1 / 127 of a row's largest value
    assert float((out - whole.double()).norm() / whole.double().norm()) < 2.0 ** -8


def test_captured_decode():
    B = 5
    w, (x, z, alpha, beta) = weights(), inputs(B, 8)
    tokens = [[t[:, i].contiguous() for t in (x, z, alpha, beta)] for i in range(8)]
    start = torch.randn((B, H, DV, DK), generator=torch.Generator().manual_seed(9)).to(DEV)
    h, want = start.clone(), []
    for i, token in enumerate(tokens):
        want.append(step(*token, h, torch.full((B,), i, device=DEV), w))
    held, at, state = [t.clone() for t in tokens[0]], torch.zeros(B, dtype=torch.int64, device=DEV), start.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held, state, at, w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(*held, state, at, w)
    state.copy_(start)
    for i, token in enumerate(tokens):
        for a, b in zip(held, token):
            a.copy_(b)
        at.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]), i
    assert torch.equal(state, h)


class Rounded(torch.autograd.Function):
    """A tensor that is stored in bf16, and whose gradient is."""

    @staticmethod
    def forward(ctx, x):
        return x.bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double()


def test_training_step():
    """Gradients of norms, rotation and delta rule in a chain against torch's
    differentiation of the definitions in 64 bits, with the chain's own
    roundings.  Where two computations of a value differ by 2^-15 of it, one value
    in a hundred and twenty rounds the other way and is 2^-7 off: 2^-7 / 11 in the
    mean square, less than 2^-10, for each of the eight tensors between the
    loss and an input."""
    B, T = 2, 140
    w, (_, z, alpha, beta) = weights(), inputs(B, T)
    g = torch.Generator().manual_seed(8)
    rows = torch.randn((B, T, COLS), generator=g).to(BF16).to(DEV)
    h0, dy = torch.randn((B, H, DV, DK), generator=g).to(DEV) / 4, torch.randn((B, T, H, DV), generator=g).to(BF16).to(DEV)
    positions = torch.arange(T, device=DEV).expand(B, T).contiguous()
    qr, kr, _ = rows.split([KEYS, KEYS, H * DV], -1)
    qr, kr = qr.unflatten(-1, (G, DK)), kr.unflatten(-1, (G, DK))
    q, k, v = heads(rows, w, positions)
    o, _, carry = ops.delta_rule(q, k, v, alpha, beta, h0, log_decay=True, save=True)
    do, dz, dnw, _ = ops.group_norm_backward(dy, o, w["nw"], gate=z, act="silu")
    dq, dk, dv, dalpha, dbeta, dh0 = ops.delta_rule_backward(do, q, k, v, alpha, beta, carry, h0, log_decay=True)
    dqr, dkr, dqw, dkw = ops.qk_norm_backward(dq, dk, qr, kr, w["qw"], w["kw"], positions, w["freq"], norm="l2")

    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    L = dict(q=leaf(qr), k=leaf(kr), v=leaf(v), alpha=leaf(alpha), beta=leaf(beta), h0=leaf(h0), qw=leaf(w["qw"]),
             kw=leaf(w["kw"]), nw=leaf(w["nw"]), z=leaf(z))
    angle = positions[..., None].double() * w["freq"].double()
    c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]

    def turned(x, weight):
        n = x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) * weight
        a, b = n[..., :ROT // 2], n[..., ROT // 2:ROT]
        return Rounded.apply(torch.cat([a * c - b * s, a * s + b * c, n[..., ROT:]], -1)).repeat_interleave(H // G, 2)

    Q, K = turned(L["q"], L["qw"]), turned(L["k"], L["kw"])
    S, outs = L["h0"], []
    for t in range(T):
        S = L["alpha"][:, t].exp()[..., None, None] * S
        kt = K[:, t][:, :, None]
        u = L["beta"][:, t][..., None] * (L["v"][:, t] - (S * kt).sum(-1))
        S = S + u[..., None] * kt
        outs.append((S * Q[:, t][:, :, None]).sum(-1))
    O = Rounded.apply(torch.stack(outs, 1))  # noqa: E741
    n = O / torch.sqrt((O * O).mean(-1, keepdim=True) + 1e-5) * L["nw"]
    (n * L["z"] * torch.sigmoid(L["z"]) * dy.double()).sum().backward()
    got = dict(q=dqr, k=dkr, v=dv, alpha=dalpha, beta=dbeta, h0=dh0, qw=dqw, kw=dkw, nw=dnw, z=dz)
    for name, value in got.items():
        want = L[name].grad
        err = float((value.double() - want).norm() / want.norm())
        # bf16 gradients of inputs are rounded once more
        assert err < 8 * 2.0 ** -10 + (2.0 ** -8 if value.dtype == BF16 else 0), (name, err)
