"""How exact the fp32 results of the chunked delta rule are (h_last and the
gradients of the gates and of h0), on the GPU against the recurrence in 64 bits.

Bounds.  What passes to these results is taken in three bf16 parts, each rounded
to 2^-9 of what the one before leaves: 2^-27 of the value, and the terms left out of
a product of two such are three of 2^-27.  Sums are fp32 in parts of at most a few
hundred terms, each off by 2^-24 of its size with either sign: 16 steps of 2^-24 are
more than all of them together, 2^-20 of the norm.  A chunk of one token has nothing
else.  In a longer one the inverse of its triangle has two parts, so its entries off
the diagonal are off by 2^-18 of themselves at most (the diagonal is 1, and exact),
and with them the share of w and z that passes through them, which is less than w
and z: 2^-18 of the norm."""

import pytest
import torch

from gpu_util import DEV
from quantized_recurrent_state_gdnq_amd import ops
from test_gpu_delta_rule import inputs, reference

pytestmark = pytest.mark.gpu

NAMES = ("h", "dalpha", "dbeta", "dh0")


def off(lead, G, H, dk, dv, lengths=None, log=False):
    spans = [(b * lead[1], (b + 1) * lead[1]) for b in range(lead[0])] if lengths is None else []
    cu = None
    if lengths is not None:
        ends = torch.tensor(lengths).cumsum(0).tolist()
        spans = list(zip([0] + ends[:-1], ends))
        cu = torch.tensor([0] + ends, dtype=torch.int32, device=DEV)
    d, more = inputs(lead, G, H, dk, dv, len(spans), 3, log)
    want = reference(d, spans, log, **more)
    _, h, carry = ops.delta_rule(**d, cu_seqlens=cu, log_decay=log, save=True)
    grads = ops.delta_rule_backward(more["do"], d["q"], d["k"], d["v"], d["alpha"], d["beta"], carry, d["h0"],
                                    more["dh_last"], cu, log_decay=log)
    got = dict(zip(NAMES, (h,) + grads[3:]))
    return {n: float((x.double() - want[n].reshape(x.shape)).norm() / want[n].norm()) for n, x in got.items()}


@pytest.mark.parametrize("log", [False, True])
@pytest.mark.parametrize("G,H,dk,dv", [(2, 2, 128, 128), (1, 3, 64, 32), (2, 4, 72, 104), (1, 1, 8, 264)])
def test_single_tokens(G, H, dk, dv, log):
    far = off((70, 1), G, H, dk, dv, log=log)
    assert max(far.values()) <= 2.0 ** -20, far
    far = off((70,), G, H, dk, dv, lengths=[1, 0] * 70, log=log)
    assert max(far.values()) <= 2.0 ** -20, far


@pytest.mark.parametrize("lead,lengths,G,H,dk,dv", [
    ((3, 64), None, 2, 4, 128, 128), ((2, 333), None, 1, 2, 64, 64), ((1, 500), None, 2, 2, 120, 136),
    ((400,), [7, 64, 0, 200, 129], 2, 4, 128, 64)])
def test_chunks(lead, lengths, G, H, dk, dv):
    far = off(lead, G, H, dk, dv, lengths)
    assert max(far.values()) <= 2.0 ** -18, far
