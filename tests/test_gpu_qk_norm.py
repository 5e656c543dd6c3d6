"""Norms of queries and keys with the position rotation (gdnq_qk_norm) on the
GPU against their definition in 64 bits.

Bounds, u = 2^-24.  A row's sum of squares is taken in parts of eight and a tree
of up to six additions: off by 15 u of itself; the mean, eps, root and division
add 5 u, half of the sum's error goes into the root: rstd is off by 13 u, n = x
rstd weight by 16 u of itself.  An angle is exact to 64 bits, its remainder in
[-pi, pi] is rounded once (at most 2^-23 = 2 u absolute) and sine and cosine add
2 u: 4 u absolute.  So a turned value a cos -+ b sin is off by (16 + 4 + 3) u (|a| +
|b|).  Back: dy turned is off by 7 u (|da| + |db|) =: 7 u T; d = dy w by one more;
the inner sum of d hat, parts of eight and a tree, by (15 + 8 + 16) u of the mean of
T w |hat|; dx = rstd (d - hat inner) follows.  A weight's gradient sums R heads
terms, each off by 24 u of T |hat|, in any order: (R heads + 24) u of the sum of
magnitudes.  bf16 results add half a step, 2^-8."""

import math

import pytest
import torch

from gpu_util import DEV, Guarded
from quantized_recurrent_state_gdnq_amd import _lib, ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32


def rotated(x, angle, interleaved, sign=1.0):
    """x [N,H,D] in 64 bits; angle [N,r/2] or None.  The second result: |a| + |b|
    of the pairs, the value itself elsewhere."""
    if angle is None:
        return x, x.abs()
    r = 2 * angle.shape[-1]
    c, s = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
    y, size = x.clone(), x.abs()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def reference(x, w, angle, norm, eps, interleaved, dy=None):
    D = x.shape[-1]
    x = x.double()
    w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    scale = 1.0 / D if norm == "rms" else 1.0
    rstd = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) * scale + eps)
    hat = x * rstd
    y, size = rotated(hat * w, angle, interleaved)
    out = {"y": (y, 23 * U * size)}
    if dy is not None:
        d0, t = rotated(dy.double(), angle, interleaved, -1.0)
        d, t_w = d0 * w, t * w.abs()
        inner = (d * hat).sum(-1, keepdim=True) * scale
        inner_e = 39 * U * (t_w * hat.abs()).sum(-1, keepdim=True) * scale
        dx = rstd * (d - hat * inner)
        out["dx"] = (dx, rstd * (8 * U * t_w + hat.abs() * inner_e + 32 * U * (d.abs() + (hat * inner).abs())))
        n = x.shape[0] * x.shape[1]
        out["dw"] = ((d0 * hat).sum((0, 1)), (n + 24) * U * (t * hat.abs()).sum((0, 1)))
    return out


def near(got, want, what):
    value, bound = want
    err = (got.double() - value).abs()
    allowed = bound + HALF[got.dtype] * value.abs() * (1 + 2.0 ** -7) + 1e-38
    assert (err <= allowed).all(), (what, float((err / allowed).max()))


def make(N, Hq, Hk, D, r, dtype, weights, far, seed=0, fused=False, pos=torch.int64):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    if fused:
        rows = n(N, (Hq + 2 * Hk) * D + 5).to(dtype).to(DEV)
        q, k = rows[:, 3:3 + Hq * D].unflatten(-1, (Hq, D)), rows[:, 3 + Hq * D:3 + (Hq + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = n(N, Hq, D).to(dtype).to(DEV), n(N, Hk, D).to(dtype).to(DEV)
    d = dict(q=q, k=k)
    if weights:
        d.update(q_weight=(1 + 0.2 * n(D)).to(DEV), k_weight=(1 + 0.2 * n(D)).to(DEV))
    if r:
        d["positions"] = torch.randint(-far if far > 2 ** 20 else 0, far, (N,), generator=g).to(pos).to(DEV)
        d["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().to(DEV)
    more = dict(dq_out=n(N, Hq, D).to(dtype).to(DEV), dk_out=n(N, Hk, D).to(dtype).to(DEV))
    return d, more


def check(d, more, norm="rms", eps=1e-6, interleaved=False):
    form = dict(norm=norm, eps=eps, interleaved=interleaved)
    q, k = ops.qk_norm(**d, **form)
    grads = ops.qk_norm_backward(**more, **d, **form)
    angle = None
    if d.get("positions") is not None:
        angle = (d["positions"].reshape(-1, 1).double() * d["inv_freq"].double())
    flat = lambda x: x.reshape((-1,) + x.shape[-2:])  # noqa: E731
    for x, dy, w, y, dx, dw, n in ((d["q"], more["dq_out"], d.get("q_weight"), q, grads[0], grads[2], "q"),
                                   (d["k"], more["dk_out"], d.get("k_weight"), k, grads[1], grads[3], "k")):
        want = reference(flat(x), w, angle, norm, eps, interleaved, flat(dy))
        near(flat(y), want["y"], n)
        near(flat(dx), want["dx"], "d" + n)
        if w is None:
            assert dw is None
        else:
            near(dw, want["dw"], n + " weight")


SIZES = [(1, 1, 1, 64, 64), (5, 2, 1, 128, 128), (3, 1, 1, 1, 0), (7, 3, 2, 2, 2), (9, 4, 4, 128, 32), (4, 2, 2, 90, 38),
         (6, 1, 3, 256, 64), (2, 2, 1, 512, 512), (5, 2, 2, 136, 8), (8, 1, 1, 64, 48), (3, 5, 2, 200, 200), (2, 1, 1, 257, 256),
         (3, 2, 2, 72, 16), (2, 2, 2, 8, 8), (11, 1, 1, 33, 30)]


@pytest.mark.parametrize("N,Hq,Hk,D,r", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(N, Hq, Hk, D, r, dtype, interleaved):
    d, more = make(N, Hq, Hk, D, r, dtype, True, 5000, seed=D)
    check(d, more, interleaved=interleaved)
    check(d, more, norm="l2", eps=1e-5, interleaved=interleaved)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_forms(fused, weights):
    for dtype in (F32, BF16):
        d, more = make(50, 4, 2, 64, 32, dtype, weights, 1000, fused=fused)
        check(d, more)


def test_aligned_rows_of_a_projection():
    rows = torch.randn(20, 8 * 128, device=DEV, dtype=BF16)
    q, k = rows[:, :4 * 128].unflatten(-1, (4, 128)), rows[:, 4 * 128:6 * 128].unflatten(-1, (2, 128))
    d, more = make(20, 4, 2, 128, 128, BF16, True, 1000)
    d.update(q=q, k=k)
    check(d, more)
    lead = {n: x.unflatten(0, (4, 5)) for n, x in d.items() if n in ("q", "k", "positions")}
    got = ops.qk_norm(**{**d, **lead})
    assert got[0].shape == (4, 5, 4, 128) and got[0].is_contiguous()
    assert all(torch.equal(a.flatten(0, 1), b) for a, b in zip(got, ops.qk_norm(**d)))


@pytest.mark.parametrize("rows", [2000, 20000])
def test_many_rows(rows):
    d, more = make(rows, 4, 1, 128, 64, BF16, True, rows)
    check(d, more)


@pytest.mark.parametrize("pos,far", [(torch.int32, 2 ** 31 - 1), (torch.int64, 2 ** 31)])
def test_far_positions(pos, far):
    d, more = make(64, 2, 2, 64, 64, F32, False, far, pos=pos)
    check(d, more, norm="l2")


def test_small_and_large_rows():
    d, more = make(8, 1, 1, 64, 64, F32, True, 100)
    d["q"][0] = 0
    d["q"][1] *= 1e-15
    d["k"][2] *= 1e15
    check(d, more)


def test_nan_stays_in_its_row():
    d, _ = make(9, 3, 2, 128, 64, BF16, True, 100)
    clean = ops.qk_norm(**d)
    d["q"][4, 1, 100] = float("nan")
    d["k"][7, 0, 3] = float("inf")
    q, k = ops.qk_norm(**d)
    bad = torch.zeros(9, 3, dtype=torch.bool)
    bad[4, 1] = True
    assert torch.equal(q[~bad], clean[0][~bad]) and torch.isnan(q[4, 1]).all()
    bad = torch.zeros(9, 2, dtype=torch.bool)
    bad[7, 0] = True
    assert torch.equal(k[~bad], clean[1][~bad])


def test_gradients_against_differences():
    d, more = make(6, 2, 1, 24, 16, F32, True, 100)
    grads = ops.qk_norm_backward(**more, **d)
    angle = d["positions"][:, None].double() * d["inv_freq"].double()
    g = torch.Generator().manual_seed(2)

    def loss(x):
        return sum(float((reference(x[n], x[n + "_weight"], angle, "rms", 1e-6, False)["y"][0] * more[f"d{n}_out"].double()).sum())
                   for n in ("q", "k"))

    for name, grad in zip(("q", "k", "q_weight", "k_weight"), grads):
        way = torch.randn(d[name].shape, generator=g, dtype=torch.float64).to(DEV)
        up, down = [loss({**{n: d[n].double() for n in ("q", "k", "q_weight", "k_weight")}, name: d[name].double() + s * way})
                    for s in (1e-5, -1e-5)]
        got, slope = float((grad.double() * way).sum()), (up - down) / 2e-5
        assert abs(got - slope) <= 64 * U * float((grad.double() * way).abs().sum()) * 4 + 1e-7 * (1 + abs(slope)), (name, got, slope)


def test_writes_stay_inside():
    d, more = make(7, 3, 2, 90, 38, BF16, True, 100)
    bufs = {n: Guarded(s, t) for n, s, t in (("q_out", (7, 3, 90), BF16), ("k_out", (7, 2, 90), BF16))}
    ops.qk_norm(**d, **{n: b.t for n, b in bufs.items()})
    back = {n: Guarded(s, t) for n, s, t in (("dq", (7, 3, 90), BF16), ("dk", (7, 2, 90), BF16), ("dq_weight", (90,), F32),
                                             ("dk_weight", (90,), F32))}
    ops.qk_norm_backward(**more, **d, **{n: b.t for n, b in back.items()})
    torch.cuda.synchronize()
    for b in (bufs | back).values():
        assert b.guards_intact() and torch.isfinite(b.t).all()


def test_same_bits_and_workspace():
    d, more = make(5000, 4, 2, 128, 64, BF16, True, 5000)
    first = ops.qk_norm_backward(**more, **d)
    ws = torch.empty(ops.qk_norm_workspace_size(d["q"], d["k"], 64), dtype=torch.uint8, device=DEV).fill_(255)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, ops.qk_norm_backward(**more, **d, workspace=ws)))
    with pytest.raises(_lib.GdnqError, match="WORKSPACE"):
        ops.qk_norm_backward(**more, **d, workspace=ws[:64])


def test_graph_replays():
    d, more = make(70, 4, 2, 128, 64, BF16, True, 1000)
    work = lambda: ops.qk_norm(**d) + ops.qk_norm_backward(**more, **d)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for i in range(4):
        new, newmore = make(70, 4, 2, 128, 64, BF16, True, 1000, seed=i + 1)
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


def test_empty():
    d, more = make(0, 2, 1, 64, 32, F32, True, 10)
    q, k = ops.qk_norm(**d)
    assert q.shape == (0, 2, 64)
    grads = ops.qk_norm_backward(**more, **d)
    assert torch.equal(grads[2], torch.zeros(64, device=DEV)) and torch.equal(grads[3], torch.zeros(64, device=DEV))


def test_refusals():
    d, more = make(6, 2, 1, 64, 32, F32, True, 10)
    bad = [dict(q=d["q"].half()), dict(k=d["k"].bfloat16()), dict(k=d["k"][:3]), dict(q=d["q"].transpose(1, 2)),
           dict(q=d["q"][..., ::2], k=d["k"][..., ::2]), dict(positions=None), dict(positions=d["positions"].float()),
           dict(positions=d["positions"][:2]), dict(inv_freq=d["inv_freq"].double()), dict(norm="mean"), dict(q=d["q"].cpu()),
           dict(q_weight=d["q_weight"][:9]), dict(q_out=d["k"]), dict(k=None)]
    for kw in bad:
        with pytest.raises(ValueError):
            ops.qk_norm(**{**d, **kw})
    with pytest.raises(_lib.GdnqError, match="SHAPE"):
        ops.qk_norm(d["q"], d["k"], positions=d["positions"], inv_freq=torch.ones(33, device=DEV))
    with pytest.raises(_lib.GdnqError, match="ALIAS"):
        ops.qk_norm(**d, q_out=d["q"])
    with pytest.raises(_lib.GdnqError, match="SHAPE"):
        ops.qk_norm(**d, eps=math.nan)
    with pytest.raises(ValueError):
        ops.qk_norm_backward(more["dq_out"][:, :1], more["dk_out"], **d)
