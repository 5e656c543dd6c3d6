"""Bad values of one sequence (gdnq_scan_*) never reach another, wherever they
stand beside the border between them: a NaN or an infinity among one
sequence's gates, inputs or gradients leaves every output of the others as it
was, bit for bit.

Channels are independent, so every channel holds one bad value, at a place of
its own: up to 130 tokens before and behind each border, in the same run of
tokens, in the same chunk (128 tokens backward, 256 forward) and in the next."""

import numpy as np
import pytest
import torch

from gpu_util import DEV
from quantized_recurrent_state_gdnq_amd import ops

pytestmark = pytest.mark.gpu

NEAR = (-131, -60, -20, -2, -1, 0, 1, 9, 20, 60, 130)


def places(bounds):
    n = bounds[-1]
    return sorted({b + d for b in bounds for d in NEAR if 0 <= b + d < n})


def both(x, gate, dy, h0, dh, cu, form):
    y, h, carry = ops.gated_scan(x, gate, h0, cu, save=True, **form)
    dx, dgate, dh0 = ops.gated_scan_backward(dy, x, gate, carry, h0, dh, cu, **form)
    return dict(y=y, dx=dx, dgate=dgate), dict(h=h, dh0=dh0)


def run(bounds, dtype, logits, lerp, odd, uniform=None, at=None):
    at = places(bounds) if at is None else at
    C = len(at) + (len(at) + odd) % 2
    n, B = bounds[-1], len(bounds) - 1
    g = torch.Generator().manual_seed(n + C)
    z = torch.randn((n, C), generator=g) * 0.8 + 2.5
    gate = (z if logits else torch.sigmoid(z)).to(dtype).to(DEV)
    x, dy = [torch.randn((n, C), generator=g).to(dtype).to(DEV) for _ in range(2)]
    h0, dh = [torch.randn((B, C), generator=g).to(DEV) for _ in range(2)]
    cu = None if uniform else torch.tensor(bounds, dtype=torch.int32, device=DEV)
    shape = (B, uniform, C) if uniform else (n, C)
    form = dict(logits=logits, lerp=lerp)

    def call(**bad):
        a = dict(x=x, gate=gate, dy=dy)
        for name, value in bad.items():
            a[name] = a[name].clone()
            a[name][at, range(len(at))] = value
        return both(*(a[k].view(shape) for k in ("x", "gate", "dy")), h0, dh, cu, form)
    seq = np.searchsorted(bounds, np.arange(n), side="right") - 1
    mine = np.searchsorted(bounds, at, side="right") - 1
    token = torch.from_numpy(seq[:, None] != mine[None]).to(DEV)  # [n, places]: of another sequence
    state = torch.from_numpy(np.arange(B)[:, None] != mine[None]).to(DEV)
    rows, states = call()
    assert all(torch.isfinite(t).all() for t in (*rows.values(), *states.values()))
    k = len(at)
    for name in ("gate", "x", "dy"):
        for value in (float("nan"), float("inf"), float("-inf")):
            bad_rows, bad_states = call(**{name: value})
            for kind, good, bad, other in (("row", rows, bad_rows, token), ("state", states, bad_states, state)):
                for key in good:
                    a, b = good[key].view(-1, C), bad[key].view(-1, C)
                    off = (a[:, :k] != b[:, :k]) & other  # a NaN differs from every value
                    where = [] if not off.any() else off.nonzero()[0].tolist()
                    assert not where, (f"{name} = {value}: {int(off.sum())} values of {key} in other sequences, the "
                                       f"first at {kind} {where[0]} for the bad token {at[where[1]]}")
                    assert torch.equal(a[:, k:], b[:, k:])
            if name == "gate" and value != value:
                last = bad_rows["y"].view(-1, C)[at, range(k)]
                assert torch.isnan(last).all()  # the bad value itself was used


FORMS = [(False, False), (True, False), (False, True), (True, True)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("logits,lerp", FORMS)
def test_packed(logits, lerp, odd, dtype):
    # borders in the middle of chunks, in neighbouring runs, next to empty and single-token sequences; a sequence of 18
    # forward chunks behind one, and borders in the chunks that close a group of 16 (tokens 3840 .. 4095 forward)
    lengths = [300, 250, 3400, 40, 1, 0, 37, 4700, 129, 20, 900]
    run([0, *np.cumsum(lengths).tolist()], dtype, logits, lerp, odd)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sequences_of_equal_length(dtype):
    run([i * 1000 for i in range(6)], dtype, False, True, 0, uniform=1000)
    run([i * 77 for i in range(9)], dtype, True, True, 1, uniform=77)


@pytest.mark.parametrize("logits", [False, True])
def test_border_in_the_chunk_that_publishes_a_state(logits):
    """Chunk 255 forward (tokens 65280 .. 65535), and backward the 256th
    128-token chunk from the end, hand a whole state on."""
    n = 65400 + 66000
    back = (n + 127) // 128 * 128 - 128 * 256  # that chunk's first token
    bounds = [0, 65400, back + 50, n]
    run(bounds, torch.float32, logits, False, 0, at=[p for p in places(bounds) if 65000 < p < n - 200])
