"""A recurrent layer as its operators are used together: the gated scan over
channels, the gated norm of its heads and the output projection in
microscaled 4 bits, for a prefill and for the decode steps that continue it,
and the same norm and projection behind the matrix-state mixer."""

import pytest
import torch

from gpu_util import DEV
import workloads as wl
from quantized_recurrent_state_gdnq_amd import ops

pytestmark = pytest.mark.gpu


def layer(x, gate, z, h0, w, wc, ws):
    """[B,T,C] inputs: y [B,T,cols], and the states after the last token."""
    B, T, C = x.shape
    h, last = ops.gated_scan(x, gate, h0, logits=True, lerp=True)
    n = ops.group_norm(h.view(B, T, -1, 64), w, gate=z.view(B, T, -1, 64), act="silu")
    return ops.mx_linear(n.view(B, T, C), wc, ws), last


def layer_step(x, gate, z, h, w, wc, ws):
    B, C = x.shape
    y = ops.gated_scan_step(x, gate, h, logits=True, lerp=True)
    n = ops.group_norm(y.view(B, -1, 64), w, gate=z.view(B, -1, 64), act="silu")
    return ops.mx_linear(n.view(B, C), wc, ws)


def plain(x, gate, z, h, w, W):
    """The layer in float64 with the roundings the operators state: the scan's
    and the norm's outputs to bf16."""
    a = torch.sigmoid(gate.double())
    hs = []
    for t in range(x.shape[1]):
        h = a[:, t] * h + torch.sigmoid(-gate[:, t].double()) * x[:, t].double()
        hs.append(h)
    y = torch.stack(hs, 1).bfloat16().double().unflatten(-1, (-1, 64))
    n = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5) * w.double()
    zz = z.double().view_as(n)
    return (n * zz * torch.sigmoid(zz)).flatten(-2).bfloat16(), h


def test_prefill_then_decode():
    B, T, C, cols, steps = 3, 200, 256, 320, 4
    g = torch.Generator().manual_seed(5)
    x, z = [torch.randn((B, T + steps, C), generator=g).bfloat16() for _ in range(2)]
    gate = (torch.randn((B, T + steps, C), generator=g) + 3).bfloat16()
    h0 = torch.randn((B, C), generator=g)
    w = torch.randn(64, generator=g) * 0.2 + 1
    W = torch.randn((cols, C), generator=g) / 16
    wc, ws = ops.mx_quantize(W.to(DEV))
    d = [t.to(DEV) for t in (x, gate, z)]
    cut = lambda i, j: [t[:, i:j].contiguous() for t in d]  # noqa: E731
    whole, last_all = layer(*d, h0.to(DEV), w.to(DEV), wc, ws)
    y, h = layer(*cut(0, T), h0.to(DEV), w.to(DEV), wc, ws)
    outs = [y]
    for t in range(T, T + steps):
        outs.append(layer_step(*(v.squeeze(1) for v in cut(t, t + 1)), h, w.to(DEV), wc, ws)[:, None])
    out = torch.cat(outs, 1).float().cpu()
    n, last = plain(x, gate, z, h0.double(), w, W)
    # fp32 states are within 1e-5 of the definition's over 204 tokens (8 units
    # of 2^-24 for each of at most 1 / (1 - a) ~ 20 remembered steps)
    assert (h.double().cpu() - last).abs().max() < 1e-5
    assert (last_all.double().cpu() - last).abs().max() < 1e-5
    # a bf16 rounding of the states or the norm that falls the other way moves a value by 2^-7 of it, and its code by at
    # most one step of the 4-bit grid: the projections agree but for the few such values (one code in a few hundred)
    nc, ns = ops.mx_quantize(n.to(DEV))
    want = ops.mx_matmul(nc, ns, wc, ws).float().cpu()
    for got in (out, whole.float().cpu()):
        assert ((got - want).norm() / want.norm()) < 0.02


def test_training_step_of_the_scan_and_norm():
    """Gradients through norm and scan in a chain, fp32, against torch's
    differentiation of the definition in float64."""
    B, T, G, D = 2, 150, 3, 40
    C = G * D
    g = torch.Generator().manual_seed(6)
    x, z, dy = [torch.randn((B, T, C), generator=g) for _ in range(3)]
    gate = torch.randn((B, T, C), generator=g) + 2
    h0, w = torch.randn((B, C), generator=g), torch.randn(D, generator=g) * 0.2 + 1
    leaves = [t.double().requires_grad_() for t in (x, gate, z, h0, w)]
    a = torch.sigmoid(leaves[1])
    h, hs = leaves[3], []
    for t in range(T):
        h = a[:, t] * h + (1 - a[:, t]) * leaves[0][:, t]
        hs.append(h)
    y = torch.stack(hs, 1).view(B, T, G, D)
    n = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5) * leaves[4]
    zz = leaves[2].view(B, T, G, D)
    ((n * zz * torch.sigmoid(zz)) * dy.double().view(B, T, G, D)).sum().backward()
    X, Z, DY, GATE, H0, Wt = [t.to(DEV) for t in (x, z, dy, gate, h0, w)]
    form = dict(logits=True, lerp=True)
    y, _, carry = ops.gated_scan(X, GATE, H0, save=True, **form)
    yv, zv, dv = (t.view(B, T, G, D) for t in (y, Z, DY))
    dn, dz, dw, _ = ops.group_norm_backward(dv, yv, Wt, gate=zv, act="silu")
    dx, dgate, dh0 = ops.gated_scan_backward(dn.view(B, T, C), X, GATE, carry, H0, **form)
    # fp32 throughout: a few units of 2^-24 per step over about 1 / (1 - a) ~ 10 steps and 40 values, far below 1e-4 of each
    # gradient's size
    for got, leaf in ((dx, 0), (dgate, 1), (dz, 2), (dh0, 3), (dw, 4)):
        want = leaves[leaf].grad
        err = (got.double().cpu().view_as(want) - want).norm() / want.norm()
        assert err < 1e-4, (leaf, float(err))


def test_behind_the_matrix_state_mixer():
    """Heads of a GDN prefill, normalised, gated and projected, [B,T,H,d_v] as
    the mixer writes them."""
    d = wl.gdn_prefill(B=1, T=128, H=2, dk=128, dv=128, seed=3)
    t = lambda v, dt=None: torch.from_numpy(v).to(DEV) if dt is None else torch.from_numpy(v).to(DEV).to(dt)  # noqa: E731
    q, k, v = (t(d[n], torch.bfloat16) for n in ("q", "k", "v"))
    o, _, _ = ops.prefill_chunked(q, k, v, t(d["alpha"]), t(d["beta"]))
    z = torch.randn(o.shape, generator=torch.Generator().manual_seed(1)).to(DEV).bfloat16()
    w = torch.ones(128, device=DEV)
    n = ops.group_norm(o, w, gate=z, act="silu")
    of, zf = o.double(), z.double()
    want = of / torch.sqrt((of * of).mean(-1, keepdim=True) + 1e-5) * zf * torch.sigmoid(zf)
    # fp32 arithmetic (about 24 units of 2^-24) and one rounding to bf16
    assert ((n.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 1e-30).all()
    wc, ws = ops.mx_quantize(torch.randn((64, 256), generator=torch.Generator().manual_seed(2)).to(DEV))
    y = ops.mx_linear(n.view(1, 128, 256), wc, ws)
    assert y.shape == (1, 128, 64) and torch.isfinite(y.float()).all()
