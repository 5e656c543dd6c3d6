"""Host-only checks of gdnq_delta_*, gdnq_qk_norm_* and gdnq_int_*: bad
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


def refused(st, code, word=""):
    assert st == code, (st, L.gdnq_last_error())
    assert word in L.gdnq_last_error().decode()


# ---------------------------------------------------------------- delta rule

def delta_p(B=2, T=100, G=2, H=4, dk=64, dv=64, ind=1, outd=1, flags=0):
    return _lib.DeltaParams(B, T, G, H, dk, dv, ind, outd, flags)


def forward(p, ws_bytes=64 * MB, **kw):
    a = dict(cu=None, q=addr(1), k=addr(2), v=addr(3), alpha=addr(4), beta=addr(5), h0=addr(6), o=addr(7), h_last=addr(8),
             carry=addr(9), ws=addr(10))
    a.update(kw)
    return _lib.delta_forward(p, a["cu"], a["q"], a["k"], a["v"], a["alpha"], a["beta"], a["h0"], a["o"], a["h_last"],
                              a["carry"], a["ws"], ws_bytes, None)


def backward(p, ws_bytes=64 * MB, **kw):
    a = dict(cu=None, q=addr(1), k=addr(2), alpha=addr(4), beta=addr(5), carry=addr(9), dout=addr(11), dh_last=addr(12),
             dq=addr(13), dk=addr(14), dv=addr(15), dalpha=addr(16), dbeta=addr(17), dh0=addr(18), ws=addr(10))
    a.update(kw)
    return _lib.delta_backward(p, a["cu"], a["q"], a["k"], a["alpha"], a["beta"], a["carry"], a["dout"], a["dh_last"],
                               a["dq"], a["dk"], a["dv"], a["dalpha"], a["dbeta"], a["dh0"], a["ws"], ws_bytes, None)


def step(p, **kw):
    a = dict(q=addr(1), k=addr(2), v=addr(3), alpha=addr(4), beta=addr(5), h=addr(6), h_out=addr(6), o=addr(7))
    a.update(kw)
    return _lib.delta_step(p, a["q"], a["k"], a["v"], a["alpha"], a["beta"], a["h"], a["h_out"], a["o"], None)


@pytest.mark.parametrize("p,code", [
    (delta_p(B=-1), SHAPE), (delta_p(T=-1), SHAPE), (delta_p(G=0), SHAPE), (delta_p(H=0), SHAPE), (delta_p(G=3, H=4), SHAPE),
    (delta_p(G=4, H=2), SHAPE), (delta_p(dk=0), SHAPE), (delta_p(dk=12), SHAPE), (delta_p(dk=136), SHAPE),
    (delta_p(dv=4), SHAPE), (delta_p(dv=1032), SHAPE), (delta_p(ind=0), DTYPE), (delta_p(ind=2), DTYPE),
    (delta_p(outd=2), DTYPE), (delta_p(flags=2), FLAGS), (delta_p(B=1 << 16, T=1 << 16), SHAPE),
    (delta_p(B=1, T=2 ** 31 - 1), SHAPE), (delta_p(B=1 << 22, T=1), SHAPE), (delta_p(B=1 << 20, T=0, dv=1024), SHAPE)])
def test_delta_parameters(p, code):
    assert forward(p) == code
    assert backward(p) == code
    for back in (False, True):
        assert _lib.delta_workspace_size(p, False, back) == 0
    assert _lib.delta_carry_size(p, False) == 0


def test_delta_pointers():
    p = delta_p()
    for name in ("q", "k", "v", "alpha", "beta", "o"):
        refused(forward(p, **{name: None}), NULL, name)
    for name in ("q", "k", "alpha", "beta", "carry", "dout", "dq", "dk", "dv", "dalpha", "dbeta"):
        refused(backward(p, **{name: None}), NULL, name)
    for name in ("q", "k", "v", "alpha", "beta", "h0", "o", "h_last", "carry"):
        refused(forward(p, **{name: addr(20) + 8}), ALIGN, name)
    for name in ("dout", "dh_last", "dq", "dk", "dv", "dalpha", "dbeta", "dh0"):
        refused(backward(p, **{name: addr(20) + 8}), ALIGN, name)
    refused(forward(p, o=addr(3)), ALIAS, "overlaps")
    refused(forward(p, h_last=addr(6)), ALIAS, "overlaps")
    refused(forward(p, carry=addr(7) + 16), ALIAS, "overlaps")
    refused(backward(p, dv=addr(11)), ALIAS, "overlaps")
    refused(backward(p, dk=addr(13)), ALIAS, "overlaps")
    refused(backward(p, dh0=addr(12)), ALIAS, "overlaps")
    refused(backward(p, dbeta=addr(9) + 1024), ALIAS, "overlaps")
    refused(forward(p, cu=addr(30) + 2), ALIGN, "cu_seqlens")
    refused(forward(p, cu=addr(8)), ALIAS, "cu_seqlens")
    assert L.gdnq_delta_forward(None, *[None] * 11, 0, None) == NULL
    assert L.gdnq_delta_backward(None, *[None] * 15, 0, None) == NULL
    assert L.gdnq_delta_step(None, *[None] * 9) == NULL


@pytest.mark.parametrize("packed", [False, True])
def test_delta_workspace(packed):
    p = delta_p(B=3, T=500)
    cu = addr(30) if packed else None
    for call, back in ((forward, False), (backward, True)):
        need = _lib.delta_workspace_size(p, packed, back)
        assert need > 0
        refused(call(p, ws_bytes=need - 1, cu=cu), WORKSPACE, str(need))
        refused(call(p, ws=None, cu=cu), WORKSPACE, "workspace")
        refused(call(p, ws=addr(20) + 8, cu=cu), ALIGN, "workspace")
        refused(call(p, ws=addr(1), cu=cu), ALIAS, "workspace")


def test_delta_carry_holds_every_chunk():
    """A chunk and head: the state entering it and its 64 writes, in two bf16 parts each."""
    per = 2 * 2 * (64 * 64 + 64 * 64)
    assert _lib.delta_carry_size(delta_p(B=2, T=100), False) == 2 * 2 * 4 * per
    # packed: at most T / 64 whole chunks and a partial one for each sequence
    assert _lib.delta_carry_size(delta_p(B=5, T=100), True) == (100 // 64 + 5) * 4 * per


def test_delta_nothing_to_do():
    p = delta_p(B=0)
    assert forward(p, q=None, k=None, v=None, alpha=None, beta=None, o=None) == 0
    assert backward(p, q=None, k=None, dq=None) == 0
    assert step(delta_p(B=0, T=1), q=None) == 0


def test_delta_step():
    p = delta_p(T=1)
    refused(step(delta_p(T=2)), SHAPE, "one token")
    refused(step(delta_p(T=1, dk=264)), SHAPE, "256")
    refused(step(delta_p(T=1, ind=3)), DTYPE)
    refused(step(delta_p(T=1, B=1 << 20, H=16, G=16)), SHAPE, "too large")
    for name in ("q", "k", "v", "alpha", "beta", "h", "h_out", "o"):
        refused(step(p, **{name: None}), NULL, name)
    refused(step(p, h_out=addr(6) + 16), ALIAS, "overlaps")
    refused(step(p, h_out=addr(3)), ALIAS, "overlaps")
    refused(step(p, o=addr(3)), ALIAS, "overlaps")
    refused(step(p, o=addr(6)), ALIAS, "overlaps")
    refused(step(p, h=addr(20) + 4), ALIGN, "h")
    refused(step(p, q=addr(20) + 2), ALIGN, "q")


@pytest.mark.parametrize("B,T,H,dv,fits", [
    (1, 64 * (2 ** 20 - 1), 16, 8, True), (1, 64 * (2 ** 20 - 1) + 1, 16, 8, False),
    (2 ** 20 - 1, 0, 16, 64, True), (2 ** 20 - 1, 0, 16, 72, False), (2 ** 20, 0, 16, 8, False)])
def test_delta_launch_limit(B, T, H, dv, fits):
    """Fewer than 2^24 workgroups of 256 threads."""
    p = delta_p(B=B, T=T, G=H, H=H, dv=dv)
    if fits:
        refused(forward(p, o=addr(20) + 8), ALIGN, "o")
    else:
        refused(forward(p), SHAPE, "too large")
        refused(backward(p), SHAPE, "too large")


@pytest.mark.parametrize("H,dk,dv,fits", [
    (2 ** 18 - 1, 128, 8, True), (2 ** 18, 128, 8, False), (2 ** 15 - 1, 8, 1024, True), (2 ** 15, 8, 1024, False)])
def test_delta_offsets_inside_a_chunk(H, dk, dv, fits):
    """64 tokens of fewer than 2^25 bf16 values each are less than 2^32 bytes."""
    p = delta_p(B=1, T=64, G=H, H=H, dk=dk, dv=dv)
    if fits:
        refused(forward(p, o=addr(20) + 8), ALIGN, "o")
    else:
        refused(forward(p), SHAPE, "2^25")
        refused(backward(p), SHAPE, "2^25")
    refused(step(delta_p(B=1, T=1, G=H, H=H, dk=dk, dv=dv), o=None), NULL, "o")


# ---------------------------------------------------------------- norms of queries and keys

def qk_p(R=10, Hq=4, Hk=2, D=64, rotary=32, dtype=1, eps=1e-6, flags=0, qs=None, ks=None):
    return _lib.QkParams(R, Hq, Hk, D, rotary, dtype, eps, flags, Hq * D if qs is None else qs, Hk * D if ks is None else ks)


def qk(p, **kw):
    a = dict(q=addr(1), k=addr(2), qw=addr(3), kw=addr(4), pos=addr(5), freq=addr(6), q_out=addr(7), k_out=addr(8))
    a.update(kw)
    return _lib.qk_norm(p, a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], a["q_out"], a["k_out"], None)


def qk_backward(p, ws_bytes=64 * MB, **kw):
    a = dict(q=addr(1), k=addr(2), qw=addr(3), kw=addr(4), pos=addr(5), freq=addr(6), dq_out=addr(7), dk_out=addr(8),
             dq=addr(9), dk=addr(10), dqw=addr(11), dkw=addr(12), ws=addr(13))
    a.update(kw)
    return _lib.qk_norm_backward(p, a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], a["dq_out"], a["dk_out"], a["dq"],
                                 a["dk"], a["dqw"], a["dkw"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("p,code", [
    (qk_p(R=-1), SHAPE), (qk_p(Hq=0), SHAPE), (qk_p(Hk=0), SHAPE), (qk_p(D=0, rotary=0), SHAPE), (qk_p(D=513), SHAPE),
    (qk_p(rotary=-2), SHAPE), (qk_p(rotary=31), SHAPE), (qk_p(rotary=66), SHAPE), (qk_p(dtype=2), DTYPE),
    (qk_p(eps=-1e-6), SHAPE), (qk_p(eps=float("nan")), SHAPE), (qk_p(eps=float("inf")), SHAPE), (qk_p(flags=8), FLAGS),
    (qk_p(qs=255), SHAPE), (qk_p(ks=127), SHAPE), (qk_p(qs=2 ** 31 + 1), SHAPE), (qk_p(qs=-256), SHAPE),
    (qk_p(Hq=2 ** 31 - 1, Hk=2 ** 31 - 1), SHAPE), (qk_p(Hq=2 ** 20, Hk=1), SHAPE), (qk_p(R=2 ** 30, Hq=1, Hk=1), SHAPE)])
def test_qk_parameters(p, code):
    assert qk(p) == code
    assert qk_backward(p) == code
    assert _lib.qk_norm_workspace_size(p) == 0


@pytest.mark.parametrize("R,fits", [(2 ** 27 - 8, True), (2 ** 27 - 7, False), (2 ** 29, False)])
def test_qk_launch_limit(R, fits):
    """Fewer than 2^24 workgroups of 256 threads, eight tokens each."""
    p = qk_p(R=R, Hq=1, Hk=1, D=1, rotary=0)
    assert (_lib.qk_norm_workspace_size(p) > 0) == fits
    for st in (qk(p, pos=None, freq=None, q_out=None), qk_backward(p, pos=None, freq=None, dq=None)):
        assert st == (NULL if fits else SHAPE)


def test_qk_pointers():
    p = qk_p()
    for name, word in (("q", "q"), ("k", "k"), ("pos", "positions"), ("freq", "inv_freq")):
        refused(qk(p, **{name: None}), NULL, word)
        refused(qk_backward(p, **{name: None}), NULL, word)
    for name in ("q_out", "k_out"):
        refused(qk(p, **{name: None}), NULL, name)
        refused(qk(p, **{name: addr(20) + 8}), ALIGN, name)
    for name in ("dq_out", "dk_out", "dq", "dk"):
        refused(qk_backward(p, **{name: None}), NULL, name)
    refused(qk(qk_p(rotary=0)), SHAPE, "rotary")
    refused(qk(p, q=addr(20) + 1), ALIGN, "q and k")
    refused(qk(qk_p(dtype=0), k=addr(20) + 2), ALIGN, "q and k")
    refused(qk(p, pos=addr(20) + 2), ALIGN, "positions")
    refused(qk(qk_p(flags=4), pos=addr(20) + 4), ALIGN, "positions")
    refused(qk(p, qw=addr(20) + 4), ALIGN, "q_weight")
    refused(qk(p, q_out=addr(1)), ALIAS, "overlaps")
    refused(qk(p, k_out=addr(7) + 16), ALIAS, "overlaps")
    # between the rows of a strided q lies what is not the call's own
    refused(qk(qk_p(qs=4096), q_out=addr(1) + 512), ALIAS, "overlaps")
    refused(qk_backward(p, dq=addr(7)), ALIAS, "overlaps")
    refused(qk_backward(p, dkw=addr(11)), ALIAS, "overlaps")


def test_qk_workspace():
    p = qk_p(R=5000)
    need = _lib.qk_norm_workspace_size(p)
    assert need > 0
    refused(qk_backward(p, ws_bytes=need - 1), WORKSPACE, str(need))
    refused(qk_backward(p, ws=None), WORKSPACE, "workspace")
    q, k = (torch.empty((5000, h, 64), dtype=torch.bfloat16, device="meta") for h in (4, 2))
    assert ops.qk_norm_workspace_size(q, k, 32) == need


def test_qk_nothing_to_do():
    p = qk_p(R=0)
    assert qk(p, q=None, k=None, pos=None, freq=None, q_out=None, k_out=None) == 0
    assert qk_backward(p, q=None, k=None, dq=None, dk=None, dqw=None, dkw=None) == 0


# ---------------------------------------------------------------- 8-bit rows

def int8_p(M=5, N=9, K=64, ind=1, outd=1, flags=0):
    return _lib.Int8Params(M, N, K, ind, outd, flags)


def matmul(p, **kw):
    a = dict(a=addr(1), s=addr(2), w=addr(3), t=addr(4), bias=addr(7), y=addr(5))
    a.update(kw)
    return _lib.int8_matmul(p, a["a"], a["s"], a["w"], a["t"], a["bias"], a["y"], None)


def linear(p, ws_bytes=64 * MB, **kw):
    a = dict(x=addr(1), w=addr(3), t=addr(4), bias=addr(7), y=addr(5), ws=addr(6))
    a.update(kw)
    return _lib.int8_linear(p, a["x"], a["w"], a["t"], a["bias"], a["y"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("p,code", [
    (int8_p(M=-1), SHAPE), (int8_p(N=0), SHAPE), (int8_p(K=0), SHAPE), (int8_p(K=24), SHAPE), (int8_p(K=1 << 17), SHAPE),
    (int8_p(M=(1 << 30) + 1), SHAPE), (int8_p(N=(1 << 25) + 1), SHAPE), (int8_p(M=1 << 30, N=1024), SHAPE),
    (int8_p(outd=2), DTYPE), (int8_p(flags=1), FLAGS)])
def test_int8_parameters(p, code):
    assert matmul(p) == code
    assert linear(p) == code
    assert _lib.int8_workspace_size(p) == 0


def test_int8_depth_keeps_the_sums_in_32_bits():
    assert ((1 << 17) - 16) * 128 * 128 < 2 ** 31 <= (1 << 17) * 128 * 128
    assert _lib.int8_workspace_size(int8_p(K=(1 << 17) - 16)) > 0


def test_int8_pointers():
    p = int8_p()
    for name, word in (("a", "a_codes"), ("s", "a_scales"), ("w", "w_codes"), ("t", "w_scales"), ("y", "y")):
        refused(matmul(p, **{name: None}), NULL, word)
        refused(matmul(p, **{name: addr(20) + 8}), ALIGN, word)
    refused(matmul(p, y=addr(3)), ALIAS, "overlaps")
    refused(matmul(p, bias=addr(5) + 16), ALIAS, "bias")
    refused(matmul(p, bias=addr(20) + 4), ALIGN, "bias")
    refused(linear(p, x=None), NULL, "x")
    refused(linear(p, y=addr(1)), ALIAS, "overlaps")
    refused(linear(p, bias=addr(5)), ALIAS, "overlaps")
    refused(linear(p, ws=addr(5)), ALIAS, "overlaps")
    refused(linear(int8_p(ind=3)), DTYPE, "in_dtype")
    need = _lib.int8_workspace_size(p)
    refused(linear(p, ws_bytes=need - 1), WORKSPACE, str(need))
    refused(linear(p, ws=None), WORKSPACE, "workspace")
    assert ops.int8_workspace_size(5, 9, 64) == need
    assert matmul(int8_p(M=0), a=None, y=None) == 0 and linear(int8_p(M=0), x=None) == 0


def test_int8_quantize():
    q = _lib.int8_quantize
    refused(q(addr(1), -1, 64, 1, addr(2), addr(3), None), SHAPE, "rows")
    refused(q(addr(1), 2 ** 31 + 1, 64, 1, addr(2), addr(3), None), SHAPE, "rows")
    refused(q(addr(1), 4, 40, 1, addr(2), addr(3), None), SHAPE, "depth")
    refused(q(addr(1), 4, 64, 2, addr(2), addr(3), None), DTYPE, "dtype")
    refused(q(None, 4, 64, 1, addr(2), addr(3), None), NULL, "x")
    refused(q(addr(1), 4, 64, 1, addr(1), addr(3), None), ALIAS, "overlaps")
    refused(q(addr(1), 4, 64, 1, addr(2) + 4, addr(3), None), ALIGN, "codes")
    assert q(None, 0, 64, 1, None, None, None) == 0


# ---------------------------------------------------------------- the wrappers' own sizes

BIG = 2 ** 32 + 10


@pytest.fixture
def meta(monkeypatch):
    """Tensors of the given shape on no device, that pass for GPU tensors."""
    monkeypatch.setattr(ops, "_need", lambda t, *a, **k: t)

    def make(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")
    return make


@pytest.mark.parametrize("lead", [(1, BIG), (BIG, 1)])
def test_delta_sizes_beyond_32_bits(meta, lead):
    q, gate = meta(*lead, 1, 8), meta(*lead, 1, dtype=torch.float32)
    carry = meta(16, dtype=torch.uint8)
    for call in (lambda: ops.delta_rule(q, q, q, gate, gate), lambda: ops.delta_rule_workspace_size(q, q),
                 lambda: ops.delta_rule_backward(q, q, q, q, gate, gate, carry)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_packed_delta_and_step_sizes_beyond_32_bits(meta):
    q, gate, cu = meta(BIG, 1, 8), meta(BIG, 1, dtype=torch.float32), meta(3, dtype=torch.int32)
    for call in (lambda: ops.delta_rule(q, q, q, gate, gate, cu_seqlens=cu),
                 lambda: ops.delta_rule_workspace_size(q, q, cu),
                 lambda: ops.delta_rule_step(q, q, q, gate, gate, meta(BIG, 1, 8, 8, dtype=torch.float32))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_int8_sizes_beyond_32_bits(meta):
    few, many = meta(4, 16, dtype=torch.int8), meta(BIG, 16, dtype=torch.int8)
    scales = lambda n: meta(n, dtype=torch.float32)  # noqa: E731
    for call in (lambda: ops.int8_matmul(few, scales(4), many, scales(BIG)),
                 lambda: ops.int8_matmul(many, scales(BIG), few, scales(4)),
                 lambda: ops.int8_linear(meta(BIG, 16), few, scales(4)),
                 lambda: ops.int8_quantize(meta(1, BIG + 6)), lambda: ops.int8_workspace_size(4, BIG, 32)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_qk_sizes_beyond_32_bits():
    for lead, heads in (((BIG,), 1), ((2, BIG // 2), 1), ((1,), BIG)):
        q = torch.empty((*lead, heads, 8), dtype=torch.bfloat16, device="meta")
        with pytest.raises(ValueError, match="2\\^31"):
            ops.qk_norm_workspace_size(q, q)
