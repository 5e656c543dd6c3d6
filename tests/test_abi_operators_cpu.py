"""Host-only checks of gdnq_scan_*, gdnq_group_norm_* and gdnq_mx_*: bad
arguments are refused, with a reason, before anything is launched.

Pointers are fake addresses that the host code compares but never
dereferences; every call below fails validation or has nothing to do, so no
kernel is launched."""

import pytest
import torch

from quantized_recurrent_state_gdnq_amd import _lib, ops

L = _lib.lib
NULL, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE, FLAGS = 1, 2, 3, 4, 5, 6, 8
MB = 1 << 20


def addr(i):
    return (1 << 40) + i * (64 * MB)


def refused(st, code, word):
    assert st == code, (st, L.gdnq_last_error())
    assert word in L.gdnq_last_error().decode()


# ---------------------------------------------------------------- scan

def scan_p(B=2, T=100, C=64, dtype=1, flags=0):
    return _lib.ScanParams(B, T, C, dtype, flags)


def forward(p, ws_bytes=64 * MB, **kw):
    a = dict(cu=None, x=addr(1), gate=addr(2), h0=addr(3), y=addr(4), h_last=addr(5), carry=addr(6), ws=addr(7))
    a.update(kw)
    return _lib.scan_forward(p, a["cu"], a["x"], a["gate"], a["h0"], a["y"], a["h_last"], a["carry"], a["ws"], ws_bytes, None)


def backward(p, ws_bytes=64 * MB, **kw):
    a = dict(cu=None, x=addr(1), gate=addr(2), h0=addr(3), carry=addr(4), dy=addr(5), dh=addr(6), dx=addr(7), dg=addr(8),
             dh0=addr(9), ws=addr(10))
    a.update(kw)
    return _lib.scan_backward(p, a["cu"], a["x"], a["gate"], a["h0"], a["carry"], a["dy"], a["dh"], a["dx"], a["dg"],
                              a["dh0"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("p,code", [
    (scan_p(B=-1), SHAPE), (scan_p(T=-1), SHAPE), (scan_p(C=0), SHAPE), (scan_p(dtype=2), DTYPE), (scan_p(flags=4), FLAGS),
    (scan_p(B=1 << 16, T=1 << 16), SHAPE), (scan_p(B=1 << 16, T=1, C=1 << 16), SHAPE),
    (scan_p(B=1, T=2 ** 31 - 1, C=2 ** 31 - 1), SHAPE)])
def test_scan_parameters(p, code):
    assert forward(p) == code
    assert backward(p) == code
    assert _lib.scan_workspace_size(p, False) == 0


def test_scan_pointers():
    p = scan_p()
    for name in ("x", "gate", "y"):
        refused(forward(p, **{name: None}), NULL, name)
    for name in ("x", "gate", "dy", "carry", "dx"):
        refused(backward(p, **{name: None}), NULL, name)
    refused(backward(p, dg=None), NULL, "dgate")
    for name in ("x", "h0", "y", "h_last", "carry"):
        refused(forward(p, **{name: addr(20) + 8}), ALIGN, name)
    refused(backward(p, dh=addr(20) + 4), ALIGN, "dh_last")
    refused(forward(p, y=addr(1)), ALIAS, "overlaps")
    refused(forward(p, h_last=addr(3)), ALIAS, "overlaps")
    refused(forward(p, carry=addr(2) + 16), ALIAS, "overlaps")
    refused(backward(p, dx=addr(5)), ALIAS, "overlaps")
    refused(backward(p, dh0=addr(6)), ALIAS, "overlaps")
    refused(forward(p, cu=addr(30) + 2), ALIGN, "cu_seqlens")
    refused(forward(p, cu=addr(4)), ALIAS, "cu_seqlens")
    assert L.gdnq_scan_forward(None, *[None] * 8, 0, None) == NULL


def test_scan_workspace():
    p = scan_p(B=1, T=100000, C=256)
    need = _lib.scan_workspace_size(p, False)
    if need:
        refused(forward(p, ws_bytes=need - 1), WORKSPACE, str(need))
        refused(forward(p, ws=None), WORKSPACE, "workspace")
        refused(backward(p, ws=addr(20) + 8), ALIGN, "workspace")
    # the packed call's tokens are its seqlen, whatever the number of sequences
    assert _lib.scan_workspace_size(scan_p(B=7, T=100000, C=256), True) == need


def test_scan_nothing_to_do():
    assert forward(scan_p(B=0), x=None, gate=None, y=None) == 0
    assert backward(scan_p(B=0), x=None) == 0


def test_scan_step():
    def step(p, **kw):
        a = dict(x=addr(1), gate=addr(2), h=addr(3), h_out=addr(3), y=addr(5))
        a.update(kw)
        return _lib.scan_step(p, a["x"], a["gate"], a["h"], a["h_out"], a["y"], None)
    p = scan_p(T=1)
    refused(step(scan_p(T=2)), SHAPE, "one token")
    for name in ("x", "gate", "h", "h_out", "y"):
        refused(step(p, **{name: None}), NULL, name)
    refused(step(p, h_out=addr(3) + 16), ALIAS, "overlaps")
    refused(step(p, y=addr(1)), ALIAS, "overlaps")
    refused(step(p, h_out=addr(2)), ALIAS, "overlaps")
    refused(step(p, h=addr(9) + 4), ALIGN, "h")
    assert step(scan_p(B=0, T=1)) == 0


# ---------------------------------------------------------------- group norm

def norm_p(R=10, G=4, D=64, dtype=1, act=1, eps=1e-5, flags=0):
    return _lib.NormParams(R, G, D, dtype, act, eps, flags)


def norm(p, **kw):
    a = dict(x=addr(1), gate=addr(2), w=addr(3), b=addr(4), y=addr(5))
    a.update(kw)
    return _lib.group_norm(p, a["x"], a["gate"], a["w"], a["b"], a["y"], None)


def norm_backward(p, ws_bytes=64 * MB, **kw):
    a = dict(x=addr(1), gate=addr(2), w=addr(3), b=addr(4), dy=addr(5), dx=addr(6), dg=addr(7), dw=addr(8), db=addr(9), ws=addr(10))
    a.update(kw)
    return _lib.group_norm_backward(p, a["x"], a["gate"], a["w"], a["b"], a["dy"], a["dx"], a["dg"], a["dw"], a["db"], a["ws"],
                                    ws_bytes, None)


@pytest.mark.parametrize("p,code", [
    (norm_p(R=-1), SHAPE), (norm_p(G=0), SHAPE), (norm_p(D=0), SHAPE), (norm_p(D=16385), SHAPE), (norm_p(dtype=5), DTYPE),
    (norm_p(act=3), FLAGS), (norm_p(act=-1), FLAGS), (norm_p(act=0), FLAGS), (norm_p(flags=4), FLAGS), (norm_p(eps=-1e-5), SHAPE),
    (norm_p(eps=float("nan")), SHAPE), (norm_p(eps=float("inf")), SHAPE), (norm_p(R=1 << 20, G=1 << 12), SHAPE)])
def test_norm_parameters(p, code):
    assert norm(p) == code
    assert norm_backward(p) == code


def test_norm_pointers():
    p = norm_p()
    refused(norm(p, x=None), NULL, "x")
    refused(norm(p, y=None), NULL, "y")
    refused(norm_backward(p, dy=None), NULL, "dy")
    refused(norm_backward(p, dx=None), NULL, "dx")
    refused(norm_backward(p, dg=None), NULL, "dgate")
    refused(norm_backward(p, gate=None), NULL, "dgate")
    refused(norm(p, w=addr(20) + 4), ALIGN, "weight")
    refused(norm(p, y=addr(1)), ALIAS, "overlaps")
    refused(norm(p, y=addr(2) - 16), ALIAS, "overlaps")
    refused(norm_backward(p, dg=addr(2)), ALIAS, "overlaps")
    refused(norm_backward(p, db=addr(8)), ALIAS, "overlaps")
    need = _lib.group_norm_workspace_size(p)
    assert need > 0
    refused(norm_backward(p, ws_bytes=need - 1), WORKSPACE, str(need))
    assert norm(norm_p(R=0), x=None, y=None, gate=None) == 0


# ---------------------------------------------------------------- microscaled 4-bit

def mx_p(M=5, N=9, K=64, ind=1, outd=1, flags=0):
    return _lib.MxParams(M, N, K, ind, outd, flags)


def matmul(p, ws_bytes=64 * MB, **kw):
    a = dict(a=addr(1), s=addr(2), w=addr(3), t=addr(4), y=addr(5), ws=addr(6))
    a.update(kw)
    return _lib.mx_matmul(p, a["a"], a["s"], a["w"], a["t"], a["y"], a["ws"], ws_bytes, None)


def linear(p, ws_bytes=64 * MB, **kw):
    a = dict(x=addr(1), w=addr(3), t=addr(4), y=addr(5), ws=addr(6))
    a.update(kw)
    return _lib.mx_linear(p, a["x"], a["w"], a["t"], a["y"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("p,code", [
    (mx_p(M=-1), SHAPE), (mx_p(N=0), SHAPE), (mx_p(K=0), SHAPE), (mx_p(K=48), SHAPE), (mx_p(K=(1 << 20) + 32), SHAPE),
    (mx_p(outd=2), DTYPE), (mx_p(flags=1), FLAGS), (mx_p(M=2 ** 31 - 1, K=1 << 20), SHAPE), (mx_p(N=2 ** 31 - 1, K=1 << 20), SHAPE)])
def test_mx_parameters(p, code):
    assert matmul(p) == code
    assert linear(p) == code
    assert _lib.mx_workspace_size(p) == 0


def test_mx_pointers():
    p = mx_p()
    for name, word in (("a", "a_codes"), ("s", "a_scales"), ("w", "w_codes"), ("t", "w_scales"), ("y", "y")):
        refused(matmul(p, **{name: None}), NULL, word)
    refused(matmul(p, w=addr(20) + 8), ALIGN, "w_codes")
    refused(matmul(p, y=addr(3)), ALIAS, "overlaps")
    refused(linear(p, x=None), NULL, "x")
    refused(linear(p, y=addr(1)), ALIAS, "overlaps")
    refused(linear(mx_p(ind=3)), DTYPE, "in_dtype")
    need = _lib.mx_workspace_size(p)
    refused(linear(p, ws_bytes=need - 1), WORKSPACE, str(need))
    refused(linear(p, ws=None), WORKSPACE, "workspace")
    assert matmul(mx_p(M=0), a=None, y=None) == 0 and linear(mx_p(M=0), x=None) == 0


def test_mx_quantize():
    q = _lib.mx_quantize
    refused(q(addr(1), -1, 64, 1, addr(2), addr(3), None), SHAPE, "rows")
    refused(q(addr(1), 4, 40, 1, addr(2), addr(3), None), SHAPE, "depth")
    refused(q(addr(1), 4, 64, 2, addr(2), addr(3), None), DTYPE, "dtype")
    refused(q(addr(1), 2 ** 31, 1 << 20, 1, addr(2), addr(3), None), SHAPE, "too large")
    refused(q(None, 4, 64, 1, addr(2), addr(3), None), NULL, "x")
    refused(q(addr(1), 4, 64, 1, addr(1), addr(3), None), ALIAS, "overlaps")
    refused(q(addr(1), 4, 64, 1, addr(2) + 4, addr(3), None), ALIGN, "codes")
    assert q(None, 0, 64, 1, None, None, None) == 0


# ---------------------------------------------------------------- launches

# A launch has fewer than 2^32 threads: sizes that would need more are refused,
# those just below are taken (a size of 0 bytes or tokens elsewhere keeps them
# from being launched).

@pytest.mark.parametrize("T,C,fits", [
    (128 * (2 ** 22 - 1), 64, True), (128 * (2 ** 22 - 1) + 1, 64, False), (2 ** 30, 1, False), (2 ** 29, 65, False)])
def test_scan_launch_limit(T, C, fits):
    p = scan_p(B=1, T=T, C=C)
    assert (_lib.scan_workspace_size(p, False) > 0) == fits
    if not fits:
        refused(forward(p), SHAPE, "too large")
        refused(backward(p), SHAPE, "too large")


@pytest.mark.parametrize("G,D,flags,fits", [
    (2 ** 13 - 1, 2 ** 13, 0, True), (2 ** 13, 2 ** 13, 0, False), (2 ** 20, 64, 0, False), (2 ** 20, 64, 2, True)])
def test_norm_launch_limit(G, D, flags, fits):
    p = norm_p(R=0, G=G, D=D, flags=flags)
    if fits:
        assert norm(p) == 0
    else:
        refused(norm(p), SHAPE, "2^26")
        refused(norm_backward(p), SHAPE, "2^26")


@pytest.mark.parametrize("M,N,fits", [
    (1, 2 ** 25, True), (1, 2 ** 25 + 1, False), (2 ** 30, 3 * 256, True), (2 ** 30, 4 * 256, False), (2 ** 15, 2 ** 25, False)])
def test_mx_launch_limit(M, N, fits):
    p = mx_p(M=M, N=N, K=32)
    assert (_lib.mx_workspace_size(p) > 0) == fits
    if not fits:
        assert matmul(p) == SHAPE
        assert linear(p) == SHAPE


@pytest.mark.parametrize("G,D,fits", [(8193, 8191, False), (17159, 3911, False), (8188, 8196, True)])
def test_norm_backward_launch_limit(G, D, fits):
    """Just below 2^26 weights: the launch that adds their gradients has 1024
    threads per 16 of them, rounded up."""
    assert 2 ** 26 - 16 <= G * D < 2 ** 26
    assert fits == (-(-G * D // 16) * 1024 < 2 ** 32)
    p = norm_p(R=0, G=G, D=D)
    if fits:
        assert norm(p) == 0
    else:
        refused(norm(p), SHAPE, "2^26")
        refused(norm_backward(p), SHAPE, "2^26")
        assert _lib.group_norm_workspace_size(p) == 0


def test_norm_workspace_of_shared_weights():
    """Teams that share the weights need no more rows of partial sums than the
    chip holds teams: 256 CUs, 16 waves each, 8 teams of 8 lanes a wave, 64
    values of two gradients."""
    p = norm_p(R=4, G=2 ** 20, D=64, flags=2)
    assert 0 < _lib.group_norm_workspace_size(p) <= 256 * 16 * 8 * 64 * 2 * 4
    # and no fewer than one row for own weights
    assert _lib.group_norm_workspace_size(norm_p(R=4, G=2 ** 19, D=64)) >= 2 ** 19 * 64 * 2 * 4
    assert _lib.group_norm_workspace_size(norm_p(R=1, G=2 ** 20, D=64, flags=2)) > 0


def test_norm_workspace_of_a_tensor():
    """Of either kind of weights: where groups may not have their own, of shared ones."""
    x = torch.empty((4, 2 ** 20, 64), dtype=torch.bfloat16, device="meta")
    shared = _lib.group_norm_workspace_size(norm_p(R=4, G=2 ** 20, D=64, flags=2))
    assert ops.group_norm_workspace_size(x) == shared
    x = torch.empty((4, 30, 64), dtype=torch.bfloat16, device="meta")
    assert ops.group_norm_workspace_size(x) == _lib.group_norm_workspace_size(norm_p(R=4, G=30, D=64))
