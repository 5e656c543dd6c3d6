"""The group norm with its activation (gdnq_group_norm) on the GPU against its
definition in 64 bits.

Bounds, with u = 2^-24 and sums of D values kept in at least 16 partial sums
(depth D/16 + 8, so a sum of terms is off by at most c = (D/16 + 16) u times
the sum of their magnitudes; divisions and square roots are inside the 16):
with the mean removed, x - mu is off by c mean|x| + u |x|; without it exact.
rstd is off by that error's share and c.  The bounds are carried through the
formulas by the product rule; activations cost 8 u and have slopes of at most
1.1 (1 for their second derivatives).  A bf16 output adds half a step, 2^-8."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded
from quantized_recurrent_state_gdnq_amd import _lib, ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def act_of(z, act):
    with np.errstate(over="ignore"):
        p, q = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    if act == "none":
        return z, np.ones_like(z)
    return (z * p, p * (1 + z * q)) if act == "silu" else (p, p * q)


def reference(x, gate, w, b, act, center, eps, dy=None):
    R, G, D = x.shape
    c = (D / 16 + 16) * U
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    w = np.ones((G, D)) if w is None else np.broadcast_to(w, (G, D))
    b = np.zeros((G, D)) if b is None else np.broadcast_to(b, (G, D))
    mu = mean(x) if center else 0.0
    d = x - mu
    d_e = c * mean(np.abs(x)) + U * np.abs(x) if center else 0.0 * x
    rstd = 1 / np.sqrt(mean(d * d) + eps)
    # relative: mean(d^2) moves by 2 mean(|d| d_e) + mean(d_e^2), rstd^2 times half of that
    rstd_r = c + rstd ** 2 * (mean(np.abs(d) * d_e) + mean(d_e * d_e))
    hat = d * rstd
    hat_e = rstd * d_e + (np.abs(hat) + rstd * d_e) * (rstd_r + 2 * U)
    n = hat * w + b
    n_e = np.abs(w) * hat_e + 2 * U * (np.abs(hat * w) + np.abs(b))
    z, z_e = (n, n_e) if gate is None else (gate, 0.0)
    f, df = act_of(z, act)
    f_e, df_e = 1.1 * z_e + 8 * U * (np.abs(f) + np.abs(z)) * (act != "none"), z_e + 8 * U * (1 + np.abs(z))
    if act == "none":
        f_e, df_e = z_e, 0.0 * f
    if gate is None:
        out = {"y": (f, f_e)}
    else:
        out = {"y": (n * f, np.abs(f) * n_e + (np.abs(n) + n_e) * f_e + U * np.abs(n * f))}
    if dy is None:
        return out
    dn, dn_e = (dy * df, np.abs(dy) * df_e) if gate is None else (dy * f, np.abs(dy) * f_e)
    dn_e = dn_e + U * np.abs(dn)
    dhat, dhat_e = dn * w, dn_e * np.abs(w) + U * np.abs(dn * w)
    p = dhat * hat
    p_e = dhat_e * np.abs(hat) + (np.abs(dhat) + dhat_e) * hat_e
    inner, inner_e = mean(p), mean(p_e) + c * mean(np.abs(p))
    m, m_e = (mean(dhat), mean(dhat_e) + c * mean(np.abs(dhat))) if center else (0.0, 0.0)
    s = dhat - m - hat * inner
    s_e = dhat_e + m_e + hat_e * np.abs(inner) + (np.abs(hat) + hat_e) * inner_e \
        + 4 * U * (np.abs(dhat) + np.abs(m) + np.abs(hat * inner))
    out["dx"] = (rstd * s, rstd * (s_e + (np.abs(s) + s_e) * (rstd_r + 2 * U)))
    if gate is not None:
        out["dgate"] = (dy * n * df, np.abs(dy) * (n_e * np.abs(df) + (np.abs(n) + n_e) * df_e) + 3 * U * np.abs(dy * n * df))
    for name, t, e in (("dweight", dn * hat, dn_e * np.abs(hat) + (np.abs(dn) + dn_e) * hat_e), ("dbias", dn, dn_e)):
        for shared in (False, True):
            ax = (0, 1) if shared else 0
            k = R * G if shared else R
            out[name, shared] = (t.sum(ax), e.sum(ax) + k * U * np.abs(t).sum(ax))
    return out


def check(got, want, name, dtype=torch.float32):
    value, bound = want
    g = got.double().cpu().numpy().reshape(value.shape)
    assert np.isfinite(g).all(), f"{name}: not finite"
    tol = bound + HALF[dtype] * (np.abs(value) + bound) + 1e-37
    bad = np.abs(g - value) > tol
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(g - value) / tol):.2f} of the bound"


def run_case(R, G, D, dtype, act, gate, center, shared, weight=True, bias=False, seed=0, scale=1.0, shift=0.2):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)
    x = (normal(R, G, D) * scale + shift).to(dtype)
    z = (normal(R, G, D) * 1.5).to(dtype) if gate else None
    dy = normal(R, G, D).to(dtype)
    pshape = (D,) if shared else (G, D)
    w = normal(*pshape) * 0.3 + 1 if weight else None
    b = normal(*pshape) * 0.3 if bias else None
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    f64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    form = dict(act=act, center=center, eps=1e-5)
    want = reference(f64(x), f64(z), f64(w), f64(b), act, center, 1e-5, f64(dy))
    ys, dxs = Guarded((R, G, D), dtype), Guarded((R, G, D), dtype)
    dzs = Guarded((R, G, D), dtype) if gate else None
    dws, dbs = Guarded(pshape, torch.float32), Guarded(pshape, torch.float32)
    y = ops.group_norm(to(x), to(w), to(b), to(z), y=ys.t, **form)
    dx, dz, dw, db = ops.group_norm_backward(to(dy), to(x), to(w), to(b), to(z), dx=dxs.t, dgate=dzs.t if gate else None,
                                             dweight=dws.t if weight else None, dbias=dbs.t if bias else None, **form)
    assert all(s.guards_intact() for s in (ys, dxs, dzs, dws, dbs) if s is not None)
    check(y, want["y"], "y", dtype)
    check(dx, want["dx"], "dx", dtype)
    if gate:
        check(dz, want["dgate"], "dgate", dtype)
    if weight:
        check(dw, want["dweight", shared], "dweight")
    if bias:
        check(db, want["dbias", shared], "dbias")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act,gate", [("none", False), ("silu", False), ("sigmoid", False), ("silu", True), ("sigmoid", True)])
@pytest.mark.parametrize("center", [False, True])
def test_forms(dtype, act, gate, center):
    run_case(37, 5, 64, dtype, act, gate, center, True, bias=True, seed=1)
    run_case(19, 3, 50, dtype, act, gate, center, False, bias=True, seed=2)


@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 15, 63, 64, 65, 100, 120, 127, 128, 129, 136, 255, 256, 257, 500, 512, 513, 1000,
                               1024, 1025, 2000, 2047, 2048, 2049, 4096, 4100, 5120, 8192, 8193, 16384])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_widths(D, dtype):
    run_case(5, 3, D, dtype, "silu", True, D > 2 and D % 2 == 0, D % 3 == 0, bias=True, seed=D)


@pytest.mark.parametrize("R,G", [(1, 1), (1, 7), (2, 64), (300, 1), (1000, 3), (257, 31), (4099, 2), (3, 4097)])
@pytest.mark.parametrize("shared", [False, True])
def test_rows_and_groups(R, G, shared):
    run_case(R, G, 24, torch.bfloat16, "silu", True, False, shared, bias=True, seed=R + G)
    run_case(R, G, 11, torch.float32, "silu", False, True, shared, bias=True, seed=R + G + 1)


def test_without_weights():
    run_case(30, 4, 128, torch.bfloat16, "silu", True, False, False, weight=False, seed=3)
    run_case(30, 4, 128, torch.float32, "none", False, True, False, weight=False, bias=True, seed=4)


def test_far_from_zero():
    """A mean a hundred times the spread: the variance comes from centred
    values, not from a difference of squares."""
    run_case(16, 2, 256, torch.float32, "none", False, True, True, seed=5, scale=0.01, shift=1.0)


def test_gradients_of_absent_arguments():
    """dweight and dbias may be wanted where weight and bias are 1 and 0."""
    x, dy = torch.randn(9, 4, 32, device=DEV), torch.randn(9, 4, 32, device=DEV)
    dw, db = torch.empty(4, 32, device=DEV), torch.empty(4, 32, device=DEV)
    out = ops.group_norm_backward(dy, x, dweight=dw, dbias=db, act="silu")
    one, zero = torch.ones(4, 32, device=DEV), torch.zeros(4, 32, device=DEV)
    ref = ops.group_norm_backward(dy, x, one, zero, act="silu")
    assert out[1] is None and torch.equal(out[0], ref[0]) and torch.equal(dw, ref[2]) and torch.equal(db, ref[3])


def test_constant_and_zero_groups():
    x = torch.zeros(3, 2, 64, device=DEV)
    x[1] = 4.0
    y = ops.group_norm(x, center=True)
    assert torch.equal(y, torch.zeros_like(y))
    y = ops.group_norm(x)
    assert torch.equal(y[0], torch.zeros_like(y[0])) and torch.allclose(y[1], torch.ones_like(y[1]), rtol=1e-6)


def test_nan_stays_in_its_group():
    x, z = torch.randn(50, 4, 128, device=DEV), torch.randn(50, 4, 128, device=DEV)
    dy = torch.randn(50, 4, 128, device=DEV)
    w = torch.randn(128, device=DEV)
    clean = (ops.group_norm(x, w, gate=z, act="silu"),) + ops.group_norm_backward(dy, x, w, gate=z, act="silu")[:2]
    x[20, 2, 5] = float("nan")
    z[30, 1, 9] = float("inf")
    dirty = (ops.group_norm(x, w, gate=z, act="silu"),) + ops.group_norm_backward(dy, x, w, gate=z, act="silu")[:2]
    keep = torch.ones(50, 4, dtype=torch.bool, device=DEV)
    keep[20, 2] = keep[30, 1] = False
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(dirty[0][20, 2]).all()


def test_gradients_against_differences():
    """Central differences of the fp32 forward along a direction: step 2^-7,
    so third-order terms of order 2^-14 and sums of 2,000 fp32 values."""
    g = torch.Generator().manual_seed(8)
    R, G, D = 9, 3, 70
    x, z, dy, vx, vz = [torch.randn((R, G, D), generator=g).to(DEV) for _ in range(5)]
    w, b, vw, vb = [torch.randn((G, D), generator=g).to(DEV) for _ in range(4)]
    for act, gate in (("silu", None), ("silu", z), ("sigmoid", z), ("sigmoid", None)):
        form = dict(act=act, center=True)

        def loss(x, w, b, z):
            return float((ops.group_norm(x, w, b, z, **form).double() * dy.double()).sum())
        dx, dz, dw, db = ops.group_norm_backward(dy, x, w, b, gate, **form)
        s = 2.0 ** -7
        for grad, v, i in ((dx, vx, 0), (dw, vw, 1), (db, vb, 2), (dz, vz, 3)):
            if grad is None:
                continue
            up, down = [x, w, b, gate], [x, w, b, gate]
            up[i], down[i] = up[i] + s * v, down[i] - s * v
            diff = (loss(*up) - loss(*down)) / (2 * s)
            along, size = float((grad.double() * v.double()).sum()), float((grad.double() * v.double()).abs().sum())
            assert abs(diff - along) <= 1e-3 * size, (act, i, diff, along, size)


def test_same_bits_streams_and_graph():
    R, G, D = 3000, 16, 128
    x, z, dy = [torch.randn(R, G, D, device=DEV).bfloat16() for _ in range(3)]
    w = torch.randn(D, device=DEV)

    def work():
        return (ops.group_norm(x, w, gate=z, act="silu"),) + ops.group_norm_backward(dy, x, w, gate=z, act="silu")[:3]
    first = work()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        side = work()
    again = work()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, side, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(R, G, D, device=DEV))
        dy.copy_(torch.randn(R, G, D, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))
        torch.cuda.synchronize()


def test_no_rows():
    x = torch.empty(0, 3, 16, device=DEV)
    w = torch.ones(3, 16, device=DEV)
    assert ops.group_norm(x, w).shape == x.shape
    dx, _, dw, db = ops.group_norm_backward(x, x, w, torch.zeros_like(w))
    assert dx.shape == x.shape and torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


def test_refusals():
    x, w = torch.zeros(4, 3, 16, device=DEV), torch.ones(16, device=DEV)
    for kw in (dict(weight=w[:8]), dict(weight=w.bfloat16()), dict(weight=w, bias=torch.zeros(3, 16, device=DEV)),
               dict(gate=x[:2], act="silu"), dict(gate=x.bfloat16(), act="silu"), dict(act="relu"), dict(y=x[:1]),
               dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            ops.group_norm(x, **kw)
    with pytest.raises(ValueError):
        ops.group_norm(x.half())
    with pytest.raises(ValueError):
        ops.group_norm(x.transpose(0, 2))
    with pytest.raises(ValueError):
        ops.group_norm_backward(x, x, dgate=torch.empty_like(x))
    with pytest.raises(_lib.GdnqError, match="FLAGS"):
        ops.group_norm(x, gate=torch.zeros_like(x))
    with pytest.raises(_lib.GdnqError, match="ALIAS"):
        ops.group_norm(x, y=x)
    with pytest.raises(_lib.GdnqError, match="WORKSPACE"):
        ops.group_norm_backward(torch.zeros_like(x), x, w, workspace=torch.empty(4, dtype=torch.uint8, device=DEV))
