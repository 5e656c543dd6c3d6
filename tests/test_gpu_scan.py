"""The gated linear recurrence (gdnq_scan_*) on the GPU against its definition
in 64 bits.

Bound: h_t = sum over s <= t of (product of a over s+1..t) b_s.  Every factor
and every sum in fp32 adds a relative error of at most a few units u = 2^-24
(the gate 4, a product 1, a sum 1, and one more product and sum per join of
two pieces of the sequence, less than one per token): with K = 8 units per
step, |error of h_t| <= E_t with E_t = a_t (E_{t-1} + K u H_{t-1}) + K u |b_t|,
H the same recurrence over |b|.  Gradients likewise, from the back.  A bf16
output adds half a step, 2^-8 of its value."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded
from quantized_recurrent_state_gdnq_amd import _lib, ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 8
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gates(gate, logits):
    if logits:
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-gate)), 1 / (1 + np.exp(gate))
    return gate, 1 - gate


def reference(x, gate, h0, bounds, logits, lerp, dy=None, dh_last=None):
    """Definition in float64, sequence by sequence; {name: (value, bound)}."""
    a, keep = gates(gate, logits)
    b = keep * x if lerp else x
    n, C = x.shape
    B = len(bounds) - 1
    aa, ba = np.abs(a), np.abs(b)
    r = {k: np.zeros((n, C)) for k in ("y", "ye", "ya", "before", "before_e", "before_a", "lam", "lam_e", "lam_a")}
    h_last, h_last_e = np.zeros((B, C)), np.zeros((B, C))
    dh0, dh0_e = np.zeros((B, C)), np.zeros((B, C))
    for i in range(B):
        t0, t1 = bounds[i], bounds[i + 1]
        h = np.zeros(C) if h0 is None else h0[i]
        e, H = np.zeros(C), np.abs(h)
        for t in range(t0, t1):
            r["before"][t], r["before_e"][t], r["before_a"][t] = h, e, H
            e = aa[t] * (e + K * U * H) + K * U * ba[t]
            H = aa[t] * H + ba[t]
            h = a[t] * h + b[t]
            r["y"][t], r["ye"][t], r["ya"][t] = h, e, H
        h_last[i], h_last_e[i] = h, e
        if dy is None:
            continue
        m = np.zeros(C) if dh_last is None else dh_last[i]
        e, M = np.zeros(C), np.abs(m)
        for t in range(t1 - 1, t0 - 1, -1):
            m, M = dy[t] + m, np.abs(dy[t]) + M
            e = e + K * U * M
            r["lam"][t], r["lam_e"][t], r["lam_a"][t] = m, e, M
            m, e, M = a[t] * m, aa[t] * (e + K * U * M), aa[t] * M
        dh0[i], dh0_e[i] = m, e
    out = {"y": (r["y"], r["ye"]), "h_last": (h_last, h_last_e)}
    if dy is not None:
        lam, lam_e = r["lam"], r["lam_e"]
        k = keep if lerp else 1.0
        out["dx"] = (lam * k, np.abs(k) * lam_e + K * U * np.abs(lam * k))
        d = r["before"] - x if lerp else r["before"]
        d_e = r["before_e"] + (U * (np.abs(r["before"]) + np.abs(x)) if lerp else 0.0)
        f = a * keep if logits else 1.0
        out["dgate"] = (lam * d * f, np.abs(f) * (lam_e * np.abs(d) + (np.abs(lam) + lam_e) * d_e)
                        + 2 * K * U * np.abs(lam * d * f))
        out["dh0"] = (dh0, dh0_e)
    return out


def check(got, want, name, dtype=torch.float32):
    value, bound = want
    g = got.double().cpu().numpy().reshape(value.shape)
    assert np.isfinite(g).all(), f"{name}: not finite"
    tol = bound + HALF[dtype] * (np.abs(value) + bound) + 1e-37
    bad = np.abs(g - value) > tol
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(g - value) / tol):.2f} of the "
                           f"bound at {np.unravel_index(np.argmax(np.abs(g - value) / tol), value.shape)}")


def make(shape, states, dtype, logits, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(s):
        return torch.randn(s, generator=g)
    z = normal(shape) * 0.8 + 2.5
    gate = z if logits else torch.sigmoid(z)
    x, gate, dy = normal(shape).to(dtype), gate.to(dtype), normal(shape).to(dtype)
    return x, gate, dy, normal(states), normal(states)


def np64(t):
    return t.double().numpy()


def run_case(B, T, C, dtype, logits, lerp, state, seed=0, lengths=None):
    packed = lengths is not None
    if packed:
        bounds = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        B, n = len(lengths), int(bounds[-1])
        shape = (n, C)
        cu = torch.from_numpy(bounds).to(DEV)
    else:
        bounds, shape, cu = np.arange(B + 1) * T, (B, T, C), None
        n = B * T
    x, gate, dy, h0, dh_last = make(shape, (B, C), dtype, logits, seed)
    form = dict(logits=logits, lerp=lerp)
    xg, gg, dyg = x.to(DEV), gate.to(DEV), dy.to(DEV)
    h0g, dhg = (h0.to(DEV), dh_last.to(DEV)) if state else (None, None)
    ys = Guarded(shape, dtype)
    hs = Guarded((B, C), torch.float32)
    y, h, carry = ops.gated_scan(xg, gg, h0g, cu, save=True, y=ys.t, h_last=hs.t, **form)
    y2, h2 = ops.gated_scan(xg, gg, h0g, cu, **form)  # without the states for the backward pass
    assert torch.equal(y, y2) and torch.equal(h, h2)
    dxs, dgs, d0s = Guarded(shape, dtype), Guarded(shape, dtype), Guarded((B, C), torch.float32)
    dx, dgate, dh0 = ops.gated_scan_backward(dyg, xg, gg, carry, h0g, dhg, cu, dx=dxs.t, dgate=dgs.t, dh0=d0s.t, **form)
    assert all(s.guards_intact() for s in (ys, hs, dxs, dgs, d0s))
    want = reference(np64(x).reshape(n, C), np64(gate).reshape(n, C), np64(h0) if state else None, bounds, logits, lerp,
                     np64(dy).reshape(n, C), np64(dh_last) if state else None)
    check(y, want["y"], "y", dtype)
    check(h, want["h_last"], "h_last")
    check(dx, want["dx"], "dx", dtype)
    check(dgate, want["dgate"], "dgate", dtype)
    check(dh0, want["dh0"], "dh0")


FORMS = [(False, False), (True, False), (False, True), (True, True)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("logits,lerp", FORMS)
def test_forms(dtype, logits, lerp):
    run_case(2, 300, 70, dtype, logits, lerp, True, seed=1)
    run_case(2, 131, 33, dtype, logits, lerp, False, seed=2)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 511, 2047, 2048, 2049, 4500])
def test_lengths(T):
    run_case(1, T, 64, torch.bfloat16, True, True, True, seed=T)


@pytest.mark.parametrize("C", [1, 2, 3, 63, 64, 65, 126, 127, 128, 129, 130, 255, 257, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_channels(C, dtype):
    run_case(3, 150, C, dtype, False, True, True, seed=C)


def exact(x, a, dy, h0, dh_last, bounds):
    """The recurrence and its gradients for gates of 1 and -1 and small
    integers, whose every sum and product is exact, in int64."""
    y, dx, dg = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    h_last, dh0 = h0.copy(), dh_last.copy()
    for i, (t0, t1) in enumerate(zip(bounds[:-1], bounds[1:])):
        if t0 == t1:
            continue
        p = np.cumprod(a[t0:t1], 0)
        h = p * (h0[i] + np.cumsum(p * x[t0:t1], 0))
        before = np.concatenate([h0[i][None], h[:-1]])
        d = dy[t0:t1].copy()
        d[-1] += dh_last[i]
        lam = p * np.cumsum((p * d)[::-1], 0)[::-1]
        y[t0:t1], dx[t0:t1], dg[t0:t1] = h, lam, lam * before
        h_last[i], dh0[i] = h[-1], a[t0] * lam[0]
    return dict(y=y, h_last=h_last, dx=dx, dgate=dg, dh0=dh0)


# Sequences longer than 256 chunks (65536 tokens forward, 32768 backward), that
# nothing is forgotten in: the states handed on have to be whole.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C", [1, 2, 66])
@pytest.mark.parametrize("lengths", [[33000], [70001], [140000], [10, 65700, 0, 66500, 33]])
def test_long_memory(lengths, C, dtype):
    bounds = np.concatenate([[0], np.cumsum(lengths)])
    n, B = int(bounds[-1]), len(lengths)
    rng = np.random.default_rng(n + C)
    x, dy = rng.integers(-1, 2, (n, C)), rng.integers(-1, 2, (n, C))
    a = np.where(rng.random((n, C)) < 0.001, -1, 1)
    h0, dh_last = rng.integers(-9, 10, (B, C)), rng.integers(-9, 10, (B, C))

    def gpu(v, t):
        return torch.from_numpy(v).to(DEV).to(t)
    cu = gpu(bounds, torch.int32)
    xs, gs, dys, h0s, dhs = gpu(x, dtype), gpu(a, dtype), gpu(dy, dtype), gpu(h0, torch.float32), gpu(dh_last, torch.float32)
    y, h, carry = ops.gated_scan(xs, gs, h0s, cu, save=True)
    dx, dgate, dh0 = ops.gated_scan_backward(dys, xs, gs, carry, h0s, dhs, cu)
    want = exact(x, a, dy, h0, dh_last, bounds)
    assert max(np.abs(v).max() for v in want.values()) < 2 ** 24
    for name, got, t in (("y", y, dtype), ("h_last", h, torch.float32), ("dx", dx, dtype), ("dgate", dgate, dtype),
                         ("dh0", dh0, torch.float32)):
        assert torch.equal(got.cpu(), torch.from_numpy(want[name]).float().to(t)), name


def test_batches():
    run_case(700, 3, 5, torch.float32, True, False, True, seed=3)
    run_case(33, 128, 130, torch.bfloat16, True, True, True, seed=4)


@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [5], [0, 3, 0, 128, 0, 1, 129, 0], [1] * 300, [127, 1, 128, 256, 400, 7],
                                     [0, 0, 4096, 0], [2100, 1, 2500, 0, 40]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_packed(lengths, dtype):
    run_case(0, 0, 66, dtype, True, True, True, seed=len(lengths), lengths=lengths)
    run_case(0, 0, 37, dtype, False, False, False, seed=len(lengths) + 1, lengths=lengths)


def test_rows_no_sequence_holds_stay():
    """Offsets that start behind 0 and end before T: the other rows keep
    their values, NaN in them reaches nothing."""
    T, C = 700, 130
    x, gate, dy, h0, _ = make((T, C), (2, C), torch.bfloat16, True, 9)
    bounds = [40, 300, 555]
    poison = np.r_[0:40, 555:700]
    x[poison], gate[poison], dy[poison] = float("nan"), float("nan"), float("nan")
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    y = torch.full((T, C), -7.0, dtype=torch.bfloat16, device=DEV)
    dx, dgate = y.clone(), y.clone()
    xg, gg, dyg, h0g = x.to(DEV), gate.to(DEV), dy.to(DEV), h0.to(DEV)
    y, h, carry = ops.gated_scan(xg, gg, h0g, cu, logits=True, lerp=True, save=True, y=y)
    dx, dgate, dh0 = ops.gated_scan_backward(dyg, xg, gg, carry, h0g, None, cu, logits=True, lerp=True, dx=dx, dgate=dgate)
    for t in (y, dx, dgate):
        assert (t[poison] == -7.0).all()
    want = reference(np64(x)[40:555], np64(gate)[40:555], np64(h0), [0, 260, 515], True, True, np64(dy)[40:555])
    check(y[40:555], want["y"], "y", torch.bfloat16)
    check(h, want["h_last"], "h_last")
    check(dx[40:555], want["dx"], "dx", torch.bfloat16)
    check(dgate[40:555], want["dgate"], "dgate", torch.bfloat16)
    check(dh0, want["dh0"], "dh0")


@pytest.mark.parametrize("offsets", [[0, 500, 300, 700], [-5, 100, 9000, 200], [700, 0, 700, 0]])
def test_malformed_offsets_stay_inside(offsets):
    """Unspecified results, but no access outside the buffers."""
    T, C = 700, 65
    x, gate, dy, h0, _ = make((T, C), (3, C), torch.float32, False, 10)
    cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    g = [Guarded((T, C), torch.float32) for _ in range(3)] + [Guarded((3, C), torch.float32) for _ in range(2)]
    xg, gg, h0g = x.to(DEV), gate.to(DEV), h0.to(DEV)
    _, _, carry = ops.gated_scan(xg, gg, h0g, cu, save=True, y=g[0].t, h_last=g[3].t)
    ops.gated_scan_backward(dy.to(DEV), xg, gg, carry, h0g, None, cu, dx=g[1].t, dgate=g[2].t, dh0=g[4].t)
    torch.cuda.synchronize()
    assert all(s.guards_intact() for s in g)


def test_nan_and_infinity_stay_in_their_channel_and_sequence():
    T, C = 900, 64
    lengths = [300, 250, 350]
    x, gate, dy, h0, dh = make((T, C), (3, C), torch.float32, True, 11)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    args = dict(logits=True, lerp=True)

    def both(x, gate, dy, h0):
        y, h, carry = ops.gated_scan(x, gate, h0, cu, save=True, **args)
        return (y, h) + ops.gated_scan_backward(dy, x, gate, carry, h0, dh.to(DEV), cu, **args)
    clean = both(x.to(DEV), gate.to(DEV), dy.to(DEV), h0.to(DEV))
    x[400, 7], h0[1, 9], dy[500, 20] = float("inf"), float("nan"), float("nan")
    gate[410, 30] = float("nan")
    dirty = both(x.to(DEV), gate.to(DEV), dy.to(DEV), h0.to(DEV))
    other = [c for c in range(C) if c not in (7, 9, 20, 30)]
    for a, b in zip(clean, dirty):
        rows = [slice(0, 300), slice(550, 900)] if a.shape[0] == T else [slice(0, 1), slice(2, 3)]
        for r in rows:
            assert torch.equal(a[r], b[r])
        assert torch.equal(a[:, other], b[:, other])
    assert torch.isinf(dirty[0][400, 7]) and torch.isnan(dirty[0][300:550, 9]).all()


def test_extreme_logits():
    """Infinite logits and the type's lowest value: gates of exactly 0 and 1."""
    C = 8
    gate = torch.zeros(1, 6, C)
    gate[0, 1], gate[0, 2], gate[0, 3], gate[0, 4] = float("inf"), float("-inf"), torch.finfo(torch.float32).min, 1000.0
    x = torch.arange(1, 7).float().view(1, 6, 1).expand(1, 6, C).contiguous()
    y, h = ops.gated_scan(x.to(DEV), gate.to(DEV), logits=True, lerp=True)
    want = [0.5, 0.5, 3.0, 4.0, 4.0, 5.0]
    assert torch.equal(y[0, :, 0].cpu(), torch.tensor(want))
    y, _ = ops.gated_scan(x.to(DEV), gate.to(DEV), logits=True)
    assert torch.equal(y[0, :, 3].cpu(), torch.tensor([1.0, 3.0, 3.0, 4.0, 9.0, 10.5]))


@pytest.mark.parametrize("B,C", [(1, 1), (3, 37), (64, 4096), (5, 8), (17, 1000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step(B, C, dtype):
    """The step is the scan of one token, and T steps are the scan of T."""
    for logits, lerp in FORMS:
        x, gate, _, h0, _ = make((B, 4, C), (B, C), dtype, logits, B * C)
        h = h0.to(DEV)
        keep = h.clone()
        ys = []
        for t in range(4):
            xt, gt = x[:, t].contiguous().to(DEV), gate[:, t].contiguous().to(DEV)
            out = torch.empty_like(h)
            y1 = ops.gated_scan_step(xt, gt, h, logits=logits, lerp=lerp, h_out=out)
            ys.append(ops.gated_scan_step(xt, gt, h, logits=logits, lerp=lerp))
            assert torch.equal(out, h) and torch.equal(y1, ys[-1])
        want = reference(np64(x).reshape(B * 4, C), np64(gate).reshape(B * 4, C), np64(h0), np.arange(B + 1) * 4, logits, lerp)
        check(torch.stack(ys, 1), want["y"], "y", dtype)
        check(h, want["h_last"], "h")
        assert torch.equal(keep.cpu(), h0)


def test_gradients_against_differences():
    """d(sum of y dy + h_last dh) by central differences of the fp32 forward
    in a smooth direction: the sums of the gradients along it agree to 1e-3
    (step 2^-6: third-order terms about 2^-12, fp32 sums of 2,000 values)."""
    B, T, C = 2, 130, 8
    x, gate, dy, h0, dh = make((B, T, C), (B, C), torch.float32, True, 21)
    vx, vg, _, v0, _ = make((B, T, C), (B, C), torch.float32, True, 22)
    vg = vg - 2.5
    g = [t.to(DEV) for t in (x, gate, dy, h0, dh, vx, vg, v0)]
    x, gate, dy, h0, dh, vx, vg, v0 = g
    args = dict(logits=True, lerp=True)

    def loss(x, gate, h0):
        y, h = ops.gated_scan(x, gate, h0, **args)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())
    _, _, carry = ops.gated_scan(x, gate, h0, save=True, **args)
    dx, dgate, dh0 = ops.gated_scan_backward(dy, x, gate, carry, h0, dh, **args)
    s = 2.0 ** -6
    for grad, v, which in ((dx, vx, 0), (dgate, vg, 1), (dh0, v0, 2)):
        arg = [x, gate, h0]
        up, down = list(arg), list(arg)
        up[which], down[which] = arg[which] + s * v, arg[which] - s * v
        diff = (loss(*up) - loss(*down)) / (2 * s)
        along = float((grad.double() * v.double()).sum())
        size = float((grad.double() * v.double()).abs().sum())
        assert abs(diff - along) <= 1e-3 * size, (which, diff, along, size)


def test_same_bits_every_time():
    x, gate, dy, h0, dh = make((1, 20000, 256), (1, 256), torch.bfloat16, True, 31)
    g = [t.to(DEV) for t in (x, gate, dy, h0, dh)]
    first = None
    for _ in range(4):
        y, h, carry = ops.gated_scan(g[0], g[1], g[3], logits=True, lerp=True, save=True)
        out = (y, h, carry) + ops.gated_scan_backward(g[2], g[0], g[1], carry, g[3], g[4], logits=True, lerp=True)
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams, many at a time."""
    cases = [make((2, 5000, 200), (2, 200), torch.bfloat16, True, s) for s in (41, 42)]
    cases = [[t.to(DEV) for t in c] for c in cases]

    def both(c):
        y, h, carry = ops.gated_scan(c[0], c[1], c[3], logits=True, save=True)
        return (y, h) + ops.gated_scan_backward(c[2], c[0], c[1], carry, c[3], c[4], logits=True)
    alone = [both(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(6):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(both(c))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(alone[i % 2], out))


def test_graph_replays():
    """Forward, backward and step in one captured graph, replayed between
    eager calls, on new inputs each time."""
    B, T, C = 2, 1500, 96
    x, gate, dy, h0, dh = [t.to(DEV) for t in make((B, T, C), (B, C), torch.bfloat16, True, 51)]
    args = dict(logits=True, lerp=True)
    outs = {}

    def work():
        y, h, carry = ops.gated_scan(x, gate, h0, save=True, **args)
        dx, dgate, dh0 = ops.gated_scan_backward(dy, x, gate, carry, h0, dh, **args)
        step = ops.gated_scan_step(x[:, -1].contiguous(), gate[:, -1].contiguous(), h, **args)
        outs.update(y=y, h=h, dx=dx, dgate=dgate, dh0=dh0, step=step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    captured = dict(outs)
    for seed in range(52, 56):
        new = make((B, T, C), (B, C), torch.bfloat16, True, seed)
        for a, b in zip((x, gate, dy, h0, dh), new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in captured.items()}
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], outs[k]) for k in got)


def test_empty_calls():
    z = torch.empty((0, 5, 7), device=DEV)
    y, h = ops.gated_scan(z, z)
    assert y.shape == (0, 5, 7) and h.shape == (0, 7)
    z = torch.empty((3, 0, 7), device=DEV)
    h0 = torch.randn(3, 7, device=DEV)
    y, h, carry = ops.gated_scan(z, z, h0, save=True)
    assert torch.equal(h, h0) and carry.shape == (0, 7)
    dh = torch.randn(3, 7, device=DEV)
    assert torch.equal(ops.gated_scan_backward(z, z, z, carry, h0, dh)[2], dh)
    assert torch.equal(ops.gated_scan_backward(z, z, z, carry, h0)[2], torch.zeros_like(dh))


def test_refusals():
    x = torch.zeros((2, 4, 8), device=DEV)
    h = torch.zeros((2, 8), device=DEV)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    bad = [dict(gate=x.bfloat16()), dict(gate=x[:, :3]), dict(gate=x.cpu()), dict(x=x.half(), gate=x.half()),
           dict(x=x[0], gate=x[0]), dict(cu_seqlens=cu), dict(h0=h[:1]), dict(h0=h.bfloat16()), dict(y=x[:, :2]),
           dict(x=x[0], gate=x[0], cu_seqlens=cu.long()), dict(carry=h), dict(x=x.transpose(1, 2), gate=x.transpose(1, 2))]
    for kw in bad:
        with pytest.raises(ValueError):
            ops.gated_scan(**dict(dict(x=x, gate=x), **kw))
    with pytest.raises(ValueError):
        ops.gated_scan_step(x, x, h)
    with pytest.raises(_lib.GdnqError, match="ALIAS"):
        ops.gated_scan(x, torch.zeros_like(x), y=x)
    with pytest.raises(_lib.GdnqError, match="ALIGN"):
        flat = torch.zeros(2 * 4 * 8 + 1, device=DEV)
        ops.gated_scan(x, flat[1:].view(2, 4, 8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_logits(dtype):
    """a and 1 - a alone in a state (fp32, whatever the call's type), over all
    logits whose smaller side is a normal number.  K units; in bf16 calls the
    exponent z log2(e) is a rounded product with a rounded constant (1.44269504,
    off by 0.23 u of itself), which adds 1.25 |z| units to the smaller side."""
    z = torch.linspace(-87, 87, 4096).to(dtype)
    zero, one = torch.zeros_like(z)[None], torch.ones_like(z)[None]
    state = torch.ones((1, z.numel()), device=DEV)
    a, keep = state.clone(), torch.zeros_like(state)
    ops.gated_scan_step(zero.to(DEV), z[None].to(DEV), a, logits=True)
    ops.gated_scan_step(one.to(DEV), z[None].to(DEV), keep, logits=True, lerp=True)
    v = np64(z)
    for got, want, small in ((a, 1 / (1 + np.exp(-v)), v < 0), (keep, 1 / (1 + np.exp(v)), v > 0)):
        units = K + (1.25 * np.abs(v) if dtype == torch.bfloat16 else 0.0)
        tail = np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v)))
        tol = np.where(small, units * U * want, units * U * tail + K * U)
        err = np.abs(got[0].double().cpu().numpy() - want)
        assert (err <= tol).all(), (np.max(err / tol), v[np.argmax(err / tol)])
