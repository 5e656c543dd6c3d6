"""The delta rule with its state in fp32 (gdnq_delta_*) on the GPU against the
recurrence itself, a token at a time in 64 bits, and its gradients against the
adjoint of that recurrence and against differences.

Bounds.  A product of fp32 values takes them in two bf16 parts: the lower one is
rounded (2^-9 of at most 2^-9 of the value) and the product of two lower ones
left out (2^-18 of a term), so a term is off by at most 2^-17 of itself, with
either sign, 2^-19 in the mean square.  Such errors add up as the terms
themselves do, so a sum of terms of either sign is off by 2^-19 of its size in
the mean square; sums in fp32 add less.  A token's output passes six such
products in a chunk (K S, the inverse, M u, Q S, the update, and the state
before), the gradients twelve at most; if all erred alike, 6 x 2^-18 = 2.3e-5 and
12 x 2^-18 = 4.6e-5 of the norm of a result.  FWD and BWD are those, of the 2-norm
of the tensor; a single value may be off by 40 times that share of the root mean
square.  bf16 results add half a step, 2^-8 of the value at most.  Where the
inverse itself is large (equal keys) the bound is times its norm."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded
from quantized_recurrent_state_gdnq_amd import _lib, ops

pytestmark = pytest.mark.gpu

FWD, BWD = 6 * 2.0 ** -18, 12 * 2.0 ** -18
HALF = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def inputs(lead, G, H, dk, dv, seqs, seed=0, log=False, dtype=BF16, lean=0.5, decay=-3.0):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731

    def unit(heads):
        x = normal(*lead, heads, dk) + lean * normal(heads, dk)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    la = -torch.nn.functional.softplus(0.5 * normal(*lead, H) + decay)
    d = dict(q=unit(G), k=unit(G), v=normal(*lead, H, dv).to(dtype), alpha=la if log else la.exp(),
             beta=torch.sigmoid(normal(*lead, H)), h0=0.5 * normal(seqs, H, dv, dk))
    more = dict(do=normal(*lead, H, dv).to(BF16), dh_last=0.5 * normal(seqs, H, dv, dk))
    return {k: v.to(DEV) for k, v in d.items()}, {k: v.to(DEV) for k, v in more.items()}


def reference(d, spans, log=False, do=None, dh_last=None):
    """Per token, in 64 bits.  Arrays are flat over the tokens: [N,..]; spans
    are the sequences' tokens."""
    G, H = d["q"].shape[-2], d["v"].shape[-2]
    flat = lambda x, n: x.double().reshape((-1,) + x.shape[-n:])  # noqa: E731
    q, k = [flat(d[n], 2).repeat_interleave(H // G, 1)[:, :, None] for n in ("q", "k")]
    v, a, b = flat(d["v"], 2), flat(d["alpha"], 1), flat(d["beta"], 1)
    if log:
        a = a.exp()
    o = torch.zeros_like(v)
    out = {"o": o, "h": []}
    grads = do is not None
    if grads:
        do = flat(do, 2)
        out.update(dq=torch.zeros_like(q[:, :, 0]), dk=torch.zeros_like(k[:, :, 0]), dv=torch.zeros_like(v),
                   dalpha=torch.zeros_like(a), dbeta=torch.zeros_like(b), dh0=[])
    for s, (t0, t1) in enumerate(spans):
        h = d["h0"][s].double() if d["h0"] is not None else torch.zeros((H, v.shape[-1], q.shape[-1]), dtype=torch.float64, device=DEV)
        states, errors = [h], []
        for t in range(t0, t1):
            decayed = a[t][:, None, None] * h
            w = v[t] - (decayed * k[t]).sum(-1)
            h = decayed + (b[t][:, None] * w)[..., None] * k[t]
            o[t] = (h * q[t]).sum(-1)
            states.append(h)
            errors.append(w)
        out["h"].append(h)
        if not grads:
            continue
        dh = dh_last[s].double() if dh_last is not None else torch.zeros_like(h)
        for t in reversed(range(t0, t1)):
            before, after, w = states[t - t0], states[t - t0 + 1], errors[t - t0]
            out["dq"][t] = (after * do[t][..., None]).sum(-2)
            dh = dh + do[t][..., None] * q[t]
            du = (dh * k[t]).sum(-1)
            dw = b[t][:, None] * du
            out["dbeta"][t] = (du * w).sum(-1)
            out["dv"][t] = dw
            dk = (dh * (b[t][:, None] * w)[..., None]).sum(-2) - a[t][:, None] * (before * dw[..., None]).sum(-2)
            out["dk"][t] = dk
            dh = dh - dw[..., None] * k[t]
            out["dalpha"][t] = (dh * before).sum((-1, -2)) * (a[t] if log else 1.0)
            dh = a[t][:, None, None] * dh
        out["dh0"].append(dh)
    empty = torch.zeros((0, H, v.shape[-1], q.shape[-1]), dtype=torch.float64, device=DEV)
    for n in ("h", "dh0"):
        if n in out:
            out[n] = torch.stack(out[n]) if out[n] else empty
    if grads:
        for n in ("dq", "dk"):
            out[n] = out[n].unflatten(1, (G, -1)).sum(2)
    return out


def near(got, want, bound, what):
    want = want.reshape(got.shape)
    err = (got.double() - want).abs()
    allowed = HALF * want.abs() if got.dtype == BF16 else 0.0 * want.abs()
    over = (err - allowed).clamp_min(0)
    size = want.norm()
    assert torch.isfinite(got).all(), what
    assert float(over.norm()) <= bound * float(size) + 1e-30, (what, float(over.norm() / size), bound)
    rms = float(size) / max(1, want.numel()) ** 0.5
    assert float(over.max()) <= 40 * bound * rms + 1e-30 if over.numel() else True, (what, float(over.max()) / rms, bound)


def check(lead, G, H, dk, dv, *, lengths=None, start=0, log=False, state=True, dh=True, seed=0, scale=1.0, change=None, **kw):
    spans = []
    if lengths is None:
        spans = [(b * lead[1], (b + 1) * lead[1]) for b in range(lead[0])]
        cu = None
    else:
        at = start
        for n in lengths:
            spans.append((at, at + n))
            at += n
        cu = torch.tensor([s[0] for s in spans] + [at], dtype=torch.int32, device=DEV)
    d, more = inputs(lead, G, H, dk, dv, len(spans), seed, log, **kw)
    if change:
        change(d)
    if not state:
        d["h0"] = None
    if not dh:
        more["dh_last"] = None
    want = reference(d, spans, log, **more)
    o, h, carry = ops.delta_rule(**d, cu_seqlens=cu, log_decay=log, save=True)
    o32, h2 = ops.delta_rule(**d, cu_seqlens=cu, log_decay=log, out_dtype=F32)
    assert torch.equal(h, h2)
    names = ("dq", "dk", "dv", "dalpha", "dbeta", "dh0")
    grads = ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"],
                                    more["dh_last"], cu, log_decay=log)
    got = dict(zip(names, grads), o=o, h=h, o32=o32)
    want["o32"] = want["o"]
    if not state:
        assert got.pop("dh0") is None
    held = torch.cat([torch.arange(a, b) for a, b in spans]).to(DEV) if spans else torch.zeros(0, dtype=torch.long, device=DEV)
    for n, x in got.items():
        w = want[n]
        if n not in ("h", "dh0"):
            x = x.reshape(w.shape)[held]
            w = w[held]
        near(x, w, (FWD if n in ("o", "o32", "h") else BWD) * scale, n)


@pytest.mark.parametrize("lead,G,H,dk,dv", [
    ((1, 1), 1, 1, 64, 64), ((2, 63), 1, 2, 64, 64), ((2, 64), 2, 2, 128, 128), ((1, 65), 1, 3, 128, 64),
    ((3, 200), 2, 4, 72, 104), ((1, 130), 1, 1, 8, 8), ((1, 257), 1, 2, 128, 256), ((2, 100), 1, 1, 56, 24),
    ((1, 500), 3, 3, 120, 136)])
@pytest.mark.parametrize("log", [False, True])
def test_shapes(lead, G, H, dk, dv, log):
    check(lead, G, H, dk, dv, log=log)


@pytest.mark.parametrize("state,dh", [(False, False), (False, True), (True, False)])
def test_without_states(state, dh):
    check((2, 150), 2, 2, 64, 64, state=state, dh=dh)


@pytest.mark.parametrize("lengths", [[0, 1, 64, 0, 65, 130, 0], [200], [3] * 40, [63, 64, 65], [0, 0, 7]])
def test_packed(lengths):
    check((sum(lengths),), 2, 4, 64, 72, lengths=lengths)
    check((sum(lengths) + 9,), 1, 2, 128, 128, lengths=lengths, start=4, log=True)


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 9, (700,), generator=g).tolist()
    check((sum(lengths),), 1, 1, 64, 64, lengths=lengths)


def test_strong_decay():
    """Products of a chunk's decays far below fp32's range, next to mild ones."""
    def change(d):
        d["alpha"][:, 10:40] = 1e-12
        d["alpha"][:, 70] = 1e-20
    check((1, 200), 1, 2, 64, 64, change=change)
    check((2, 150), 1, 2, 128, 64, decay=2.0)


def test_zero_decay():
    """alpha = 0 forgets the state; its gradient is that of the product."""
    def change(d):
        d["alpha"][:, 5] = 0.0
        d["alpha"][:, 64] = 0.0
    check((1, 130), 1, 2, 64, 64, change=change)


def test_no_decay_no_write():
    def change(d):
        d["alpha"].fill_(1.0)
        d["beta"][:, ::3] = 0.0
    check((1, 150), 1, 2, 64, 64, change=change)


def test_equal_keys():
    """All keys of a head alike and beta near 1: I + At B is ones below the
    diagonal, its inverse is bidiagonal, of norm at most 2."""
    def change(d):
        d["k"][:] = d["k"][:, :1]
        d["beta"].clamp_(min=0.9)
    check((1, 200), 1, 1, 64, 64, change=change, scale=2.0)


def test_long():
    check((1, 2500), 1, 2, 128, 128, log=True)


# few heads of many tokens are cut into segments that run at once: what passes
# between them is a product more (of 64 decays near 1, so that it matters)
@pytest.mark.parametrize("G,H,dk,dv", [(32, 64, 72, 24), (64, 64, 128, 64), (16, 64, 64, 8)])
def test_segments(G, H, dk, dv):
    check((1, 2111), G, H, dk, dv, decay=-7.0, log=True, scale=2.0)


@pytest.mark.parametrize("lengths", [[0, 2500, 70, 1100], [40, 3000, 0, 1], [600, 700, 64, 900]])
def test_packed_segments(lengths):
    check((sum(lengths) + 3,), 8, 16, 64, 40, lengths=lengths, start=2, decay=-7.0, scale=2.0)


@pytest.mark.parametrize("state,dh", [(False, True), (True, False)])
def test_segments_without_states(state, dh):
    check((1, 2200), 64, 64, 16, 16, decay=-7.0, state=state, dh=dh, scale=2.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,G,H,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 6, 128, 128), (2, 1, 2, 72, 40), (2, 1, 1, 256, 8),
                                         (40, 4, 8, 128, 136), (5, 1, 1, 8, 1024), (1, 1, 1, 136, 64)])
def test_step(B, G, H, dk, dv, dtype):
    """One token in fp32: sums of dk terms in at least eight parts."""
    d, _ = inputs((B,), G, H, dk, dv, B, dtype=dtype)
    want = reference({k: v if k == "h0" else v[:, None] for k, v in d.items()}, [(b, b + 1) for b in range(B)])
    h = d.pop("h0")
    out = torch.empty_like(h)
    o = ops.delta_rule_step(**d, h=h, h_out=out)
    near(out, want["h"], 2.0 ** -21, "h")
    near(o, want["o"], 2.0 ** -20, "o")
    o2 = ops.delta_rule_step(**d, h=h, log_decay=False, out_dtype=F32)  # in place
    assert torch.equal(h, out)
    near(o2, want["o"], 2.0 ** -20, "o fp32")
    d["alpha"] = d["alpha"].log()
    want = reference({k: v[:, None] for k, v in d.items()} | {"h0": out}, [(b, b + 1) for b in range(B)], log=True)
    near(ops.delta_rule_step(**d, h=h, log_decay=True), want["o"], 2.0 ** -19, "o log")
    near(h, want["h"], 2.0 ** -19, "h log")


def test_chunked_then_steps():
    """A prompt in chunks, then tokens one at a time: as all of it at once."""
    B, T, n, G, H, dk, dv = 2, 100, 5, 1, 2, 128, 64
    d, _ = inputs((B, T + n), G, H, dk, dv, B)
    want = reference(d, [(b * (T + n), (b + 1) * (T + n)) for b in range(B)])
    h0 = d.pop("h0")
    o, h = ops.delta_rule(**{k: v[:, :T].contiguous() for k, v in d.items()}, h0=h0)
    outs = [o]
    for t in range(T, T + n):
        outs.append(ops.delta_rule_step(**{k: v[:, t].contiguous() for k, v in d.items()}, h=h)[:, None])
    near(torch.cat(outs, 1), want["o"], FWD, "o")
    near(h, want["h"], FWD, "h")


def test_state_into_the_quantized_cache():
    """The state after a prompt, quantized, is a decode state."""
    d, _ = inputs((2, 64), 2, 2, 64, 64, 2)
    _, h = ops.delta_rule(**d)
    codes, scales = ops.quantize_state(h)
    st = ops.DecodeState(codes, scales, window=8)
    t, _ = inputs((2,), 2, 2, 64, 64, 2, seed=9)
    o = st.step(t["q"], t["k"], t["v"], t["alpha"], t["beta"], out_dtype=F32)
    o2 = ops.delta_rule_step(t["q"], t["k"], t["v"], t["alpha"], t["beta"], h, out_dtype=F32)
    # a code is off by half a step of 1/127 of its row's largest value
    assert float((o - o2).norm()) <= 0.01 * float(o2.norm()) + 64 ** 0.5 * float(h.abs().amax()) / 254


def test_gradients_against_differences():
    """A central difference of the 64-bit recurrence along random directions,
    against the gradients' product with them."""
    lead, G, H, dk, dv = (1, 70), 1, 2, 16, 24
    d, more = inputs(lead, G, H, dk, dv, 1, seed=4)
    _, _, carry = ops.delta_rule(**d, save=True)
    grads = ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], more["dh_last"])
    g = torch.Generator().manual_seed(1)

    def loss(x):
        r = reference(x, [(0, 70)])
        return float((r["o"] * more["do"].double().reshape(r["o"].shape)).sum() + (r["h"] * more["dh_last"].double()).sum())

    for name, grad in zip(("q", "k", "v", "alpha", "beta", "h0"), grads):
        way = torch.randn(d[name].shape, generator=g, dtype=torch.float64).to(DEV)
        step = 1e-5
        up, down = [loss({**{k: v.double() for k, v in d.items()}, name: d[name].double() + s * way}) for s in (step, -step)]
        slope = (up - down) / (2 * step)
        got = float((grad.double() * way).sum())
        # each bf16 value of the gradient is off by 2^-8 of it at most, 2^-9.8 in the mean square
        tol = (2.0 ** -8 if grad.dtype == BF16 else 2 * BWD) * 3 * float(grad.double().norm()) + 1e-6 * abs(slope)
        assert abs(got - slope) <= tol, (name, got, slope, tol)


def test_shared_heads_add_up():
    """dq and dk of a key head are the sums over its value heads: those of
    calls with a head each."""
    d, more = inputs((1, 100), 1, 3, 64, 64, 1)
    _, _, carry = ops.delta_rule(**d, save=True)
    args = [d[n] for n in ("q", "k", "v", "alpha", "beta")]
    dq, dk, *_ = ops.delta_rule_backward(more["do"], *args, carry, d["h0"], more["dh_last"])
    one = torch.zeros((2,) + dq.shape, dtype=torch.float64, device=DEV)
    for h in range(3):
        e = {n: d[n][:, :, h:h + 1].contiguous() for n in ("v", "alpha", "beta")}
        h0, dh = d["h0"][:, h:h + 1].contiguous(), more["dh_last"][:, h:h + 1].contiguous()
        _, _, carry = ops.delta_rule(d["q"], d["k"], **e, h0=h0, save=True)
        got = ops.delta_rule_backward(more["do"][:, :, h:h + 1].contiguous(), d["q"], d["k"], **e, carry=carry, h0=h0, dh_last=dh)
        one += torch.stack(got[:2]).double()
    for a, b in ((dq, one[0]), (dk, one[1])):
        assert float((a.double() - b).norm()) <= 4 * HALF * float(b.norm())


def guarded_call(d, more, cu, log=False):
    """Forward and backward into guarded buffers; all outputs and the guards."""
    N = d["v"].shape[:-2]
    H, dv, G, dk = d["v"].shape[-2], d["v"].shape[-1], d["q"].shape[-2], d["q"].shape[-1]
    B = d["h0"].shape[0]
    bufs = {n: Guarded(shape, dtype) for n, shape, dtype in (
        ("o", N + (H, dv), BF16), ("h_last", (B, H, dv, dk), F32), ("dq", N + (G, dk), BF16), ("dk", N + (G, dk), BF16),
        ("dv", N + (H, dv), BF16), ("dalpha", N + (H,), F32), ("dbeta", N + (H,), F32), ("dh0", (B, H, dv, dk), F32))}
    view = {n: b.t for n, b in bufs.items()}
    _, _, carry = ops.delta_rule(**d, cu_seqlens=cu, log_decay=log, save=True, o=view["o"], h_last=view["h_last"])
    ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], more["dh_last"], cu,
                            log_decay=log, **{n: view[n] for n in ("dq", "dk", "dv", "dalpha", "dbeta", "dh0")})
    torch.cuda.synchronize()
    return view, bufs


def test_tokens_no_sequence_holds_stay():
    d, more = inputs((150,), 1, 2, 64, 64, 2)
    cu = torch.tensor([7, 70, 133], dtype=torch.int32, device=DEV)
    view, bufs = guarded_call(d, more, cu)
    assert all(b.guards_intact() for b in bufs.values())
    for n in ("o", "dq", "dk", "dv", "dalpha", "dbeta"):
        assert torch.isnan(torch.cat([view[n][:7], view[n][133:]])).all(), n
        assert torch.isfinite(view[n][7:133]).all(), n


@pytest.mark.parametrize("offsets", [[0, 500, 90], [-50, 20, 90], [90, 20, 0], [5, 5, 2 ** 31 - 1], [0, -1, 90]])
def test_malformed_offsets_stay_inside(offsets):
    d, more = inputs((90,), 1, 1, 64, 64, 2)
    cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    _, bufs = guarded_call(d, more, cu)
    assert all(b.guards_intact() for b in bufs.values())


def test_nan_stays_in_its_sequence_and_head():
    """... and reaches no chunk before its own."""
    d, _ = inputs((260,), 1, 2, 64, 64, 2)
    cu = torch.tensor([0, 100, 260], dtype=torch.int32, device=DEV)
    clean = ops.delta_rule(**d, cu_seqlens=cu)
    for bad in (float("nan"), float("inf")):
        e = {k: v.clone() for k, v in d.items()}
        e["v"][180, 1, 3] = bad  # second sequence, its second chunk
        o, h = ops.delta_rule(**e, cu_seqlens=cu)
        assert torch.equal(o[:164], clean[0][:164]) and torch.equal(o[:, 0], clean[0][:, 0])
        assert torch.equal(h[0], clean[1][0]) and torch.equal(h[1, 0], clean[1][1, 0])
        assert not torch.isfinite(o[180:, 1, 3]).any()
        keep = [c for c in range(64) if c != 3]  # a row of the state is its own
        assert torch.equal(o[:, 1, keep], clean[0][:, 1, keep])


def test_same_bits_every_time():
    d, more = inputs((3, 333), 2, 4, 128, 128, 3)
    args = [d[n] for n in ("q", "k", "v", "alpha", "beta")]

    def once():
        o, h, carry = ops.delta_rule(**d, save=True)
        return (o, h) + ops.delta_rule_backward(more["do"], *args, carry, d["h0"], more["dh_last"])

    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_two_streams_at_once():
    sets = [inputs((2, 300), 2, 2, 128, 128, 2, seed=s) for s in (1, 2)]

    def once(s):
        d, more = s
        o, h, carry = ops.delta_rule(**d, save=True)
        return (o, h) + ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], more["dh_last"])

    alone = [once(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(once(sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(alone[i], g))


def test_graph_replays():
    """Forward, backward and step in one captured graph, replayed between eager
    work on new inputs."""
    d, more = inputs((2, 200), 1, 2, 64, 64, 2)
    tok, _ = inputs((2,), 1, 2, 64, 64, 2, seed=5)
    tok.pop("h0")

    def work():
        o, h, carry = ops.delta_rule(**d, save=True)
        grads = ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], more["dh_last"])
        nxt = torch.empty_like(h)
        return (o, h) + grads + (ops.delta_rule_step(**tok, h=h, h_out=nxt), nxt)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for i in range(4):
        new, newmore = inputs((2, 200), 1, 2, 64, 64, 2, seed=10 + i)
        for n in d:
            d[n].copy_(new[n])
        for n in more:
            more[n].copy_(newmore[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_workspaces_given():
    d, more = inputs((2, 100), 1, 2, 64, 64, 2)
    size = ops.delta_rule_workspace_size(d["q"], d["v"])
    ws = torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)
    o, h, carry = ops.delta_rule(**d, save=True)
    o2, h2, carry2 = ops.delta_rule(**d, workspace=ws, carry=torch.empty_like(carry).fill_(255))
    assert torch.equal(o, o2) and torch.equal(h, h2)
    size = ops.delta_rule_workspace_size(d["q"], d["v"], backward=True)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)
    args = [more["do"]] + [d[n] for n in ("q", "k", "v", "alpha", "beta")]
    a = ops.delta_rule_backward(*args, carry, d["h0"], more["dh_last"])
    b = ops.delta_rule_backward(*args, carry2, d["h0"], more["dh_last"], workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(_lib.GdnqError, match="WORKSPACE"):
        ops.delta_rule(**d, workspace=ws[:100])


def test_empty_calls():
    d, more = inputs((3, 0), 1, 2, 64, 64, 3)
    o, h, carry = ops.delta_rule(**d, save=True)
    assert o.shape == (3, 0, 2, 64) and torch.equal(h, d["h0"])
    dh0 = ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], more["dh_last"])[5]
    assert torch.equal(dh0, more["dh_last"])
    d, _ = inputs((0, 5), 1, 2, 64, 64, 0)
    o, h = ops.delta_rule(**d)
    assert o.shape == (0, 5, 2, 64) and h.shape == (0, 2, 64, 64)


def test_refusals():
    d, more = inputs((2, 10), 2, 2, 64, 64, 2)
    cu = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    bad = [dict(q=d["q"].float()), dict(k=d["k"][:, :5]), dict(v=d["v"].cpu()), dict(alpha=d["alpha"].bfloat16()),
           dict(beta=d["beta"][:1]), dict(h0=d["h0"][:1]), dict(cu_seqlens=cu), dict(q=d["q"].transpose(1, 2)),
           dict(o=d["v"][:, :5]), dict(carry=d["h0"]), dict(out_dtype=torch.float16), dict(h_last=d["h0"].bfloat16())]
    for kw in bad:
        with pytest.raises(ValueError):
            ops.delta_rule(**{**d, **kw})
    with pytest.raises(_lib.GdnqError, match="ALIAS"):
        ops.delta_rule(**d, o=d["v"])
    with pytest.raises(_lib.GdnqError, match="SHAPE"):
        ops.delta_rule(*[d[n][..., :60].contiguous() for n in ("q", "k")], d["v"], d["alpha"], d["beta"])
    with pytest.raises(_lib.GdnqError, match="SHAPE"):  # heads that key heads do not divide
        ops.delta_rule(d["q"], d["k"], *[d[n][:, :, :1].contiguous() for n in ("v", "alpha", "beta")])
    _, _, carry = ops.delta_rule(**d, save=True)
    with pytest.raises(ValueError):
        ops.delta_rule_backward(more["do"].float(), *[d[n] for n in ("q", "k", "v", "alpha", "beta")], carry)
    with pytest.raises(ValueError):
        ops.delta_rule_backward(more["do"], *[d[n] for n in ("q", "k", "v", "alpha", "beta")], carry[:-1])
    with pytest.raises(ValueError):
        ops.delta_rule_step(*[d[n] for n in ("q", "k", "v", "alpha", "beta")], d["h0"])
