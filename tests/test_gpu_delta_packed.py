"""Packed sequences of very different lengths through the delta rule: the longest
start first, and those far longer than a CU's share are cut into segments; up to
64 sequences are put in order, more keep their own."""

import pytest
import torch

from gpu_util import DEV
from quantized_recurrent_state_gdnq_amd import ops
from test_gpu_delta_rule import check, guarded_call, inputs

pytestmark = pytest.mark.gpu


# 16 chunks of 64 tokens are the longest that is never cut, segments have 8 or more
@pytest.mark.parametrize("lengths", [[1024, 1025, 64, 1], [0, 1100, 0, 1100, 1100, 0], [3000], [1088, 5, 2113, 512, 513]])
@pytest.mark.parametrize("log", [False, True])
def test_lengths_around_a_cut(lengths, log):
    check((sum(lengths),), 2, 4, 64, 72, lengths=lengths, log=log, decay=-7.0, scale=2.0)


@pytest.mark.parametrize("count", [63, 64, 65, 130])
def test_many_sequences_with_a_long_one(count):
    lengths = [(7 * i) % 23 for i in range(count - 1)]
    lengths.insert(count // 2, 1500)
    check((sum(lengths) + 9,), 3, 6, 32, 24, lengths=lengths, start=4, decay=-6.0, scale=2.0)


def test_equal_lengths():
    check((12 * 70,), 2, 2, 64, 64, lengths=[70] * 12)


def test_wide_heads_of_two_sequences():
    check((2000,), 4, 8, 128, 136, lengths=[1800, 200], decay=-7.0, scale=2.0)


@pytest.mark.parametrize("offsets", [[0, 3000, 0, 3000, 0, 3000], [0, 2900, 2800, 2900, 100, 3000], [3000, 0, 2000, -7, 5000, 1]])
def test_malformed_offsets_of_long_sequences_stay_inside(offsets):
    """More cut sequences than T tokens could hold: those beyond the workspace's segments are left out."""
    d, more = inputs((3000,), 1, 2, 64, 64, 5)
    cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    _, bufs = guarded_call(d, more, cu)
    assert all(b.guards_intact() for b in bufs.values())


def test_workspace_alone_is_written():
    """Nothing behind the bytes that a call asks for, with segments in them."""
    lengths = [2500, 70, 1100]
    d, more = inputs((sum(lengths),), 2, 4, 64, 64, 3)
    cu = torch.tensor([0, 2500, 2570, 3670], dtype=torch.int32, device=DEV)
    need, need_back = [ops.delta_rule_workspace_size(d["q"], d["v"], cu, backward=back) for back in (False, True)]
    ws, ws_back = [torch.full((n + 65536,), 0xA5, dtype=torch.uint8, device=DEV) for n in (need, need_back)]
    _, _, carry = ops.delta_rule(**d, cu_seqlens=cu, save=True, workspace=ws)
    ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], cu_seqlens=cu, workspace=ws_back)
    assert (ws[need:] == 0xA5).all() and (ws_back[need_back:] == 0xA5).all()


def test_arrays_beyond_32_bits():
    """Values of more than 2^32 bytes, what is left of the chunks of more: the last
    sequence's results are, bit for bit, those of a call of its own."""
    N, n, G, H, d = 66000, 200, 2, 256, 128
    g = torch.Generator(device=DEV).manual_seed(2)
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
    q, k = [torch.nn.functional.normalize(rand(N, G, d) - 0.5, dim=-1).bfloat16() for _ in range(2)]
    v, do = [torch.empty((N, H, d), dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2)]
    alpha, beta = 1 - 0.1 * rand(N, H), rand(N, H)
    assert v.numel() * 2 > 2 ** 32

    def call(first, offsets):
        cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        a = [t[first:] for t in (q, k, v, alpha, beta)]
        o, h, carry = ops.delta_rule(*a, cu_seqlens=cu, save=True)
        grads = ops.delta_rule_backward(do[first:], *a, carry, cu_seqlens=cu)
        return [t[-n:].clone() for t in (o, *grads[:5])] + [h[-1].clone()]

    for x, y in zip(call(0, [0, N - n, N]), call(N - n, [0, n])):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def test_replayed_with_other_offsets():
    """The offsets are read on the device: a captured call follows what they hold, whatever is cut then."""
    N = 2600
    d, more = inputs((N,), 2, 4, 64, 64, 3)
    offsets = [[0, 900, 1800, N], [0, 0, 2599, N], [10, 1200, 1201, 2500], [0, 100, 164, N]]
    cu = torch.tensor(offsets[0], dtype=torch.int32, device=DEV)
    out = {n: torch.zeros_like(t) for n, t in (("o", d["v"]), ("dq", d["q"]), ("dk", d["k"]), ("dv", d["v"]),
                                               ("dalpha", d["alpha"]), ("dbeta", d["beta"]), ("dh0", d["h0"]), ("h_last", d["h0"]))}

    def call():
        _, _, carry = ops.delta_rule(**d, cu_seqlens=cu, save=True, o=out["o"], h_last=out["h_last"])
        ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"], more["dh_last"], cu,
                                **{n: out[n] for n in ("dq", "dk", "dv", "dalpha", "dbeta", "dh0")})

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for values in offsets + offsets[::-1]:
        cu.copy_(torch.tensor(values, dtype=torch.int32))
        for t in out.values():
            t.zero_()
        call()
        want = {n: t.clone() for n, t in out.items()}
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in out.items():
            assert torch.equal(t, want[n]), (values, n)
