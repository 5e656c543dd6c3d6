"""One token of the delta rule with four rows of a state in flight in a lane, the
form that calls of 1024 workgroups and more take: each width of a lane group, both
types, d_v that ends inside the last group of rows, in place and out of place."""

import pytest
import torch

from gpu_util import DEV, Guarded
from quantized_recurrent_state_gdnq_amd import ops
from test_gpu_delta_rule import BF16, F32, inputs, near, reference

pytestmark = pytest.mark.gpu


# lanes of a row (8 columns each), rows of a pass: 256 / lanes, four in flight
@pytest.mark.parametrize("B,G,H,dk,dv", [(64, 4, 8, 128, 136), (130, 1, 8, 64, 200), (70, 1, 8, 136, 72), (90, 2, 6, 72, 264),
                                         (16, 32, 64, 256, 40), (600, 2, 2, 40, 104)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_four_rows(B, G, H, dk, dv, dtype):
    rows = 256 // (8 if dk <= 64 else 16 if dk <= 128 else 32)
    assert B * H * -(-dv // (4 * rows)) >= 1024
    d, _ = inputs((B,), G, H, dk, dv, B, dtype=dtype, seed=2)
    want = reference({k: v if k == "h0" else v[:, None] for k, v in d.items()}, [(b, b + 1) for b in range(B)])
    h = d.pop("h0")
    out, o = Guarded(h.shape, F32), Guarded((B, H, dv), dtype)
    ops.delta_rule_step(**d, h=h, h_out=out.t, o=o.t)
    torch.cuda.synchronize()
    assert out.guards_intact() and o.guards_intact()
    near(out.t, want["h"], 2.0 ** -21, "h")
    near(o.t, want["o"], 2.0 ** -20, "o")
    o2 = ops.delta_rule_step(**d, h=h, out_dtype=F32)  # in place
    assert torch.equal(h, out.t)
    near(o2, want["o"], 2.0 ** -20, "o fp32")
    # a batch of few workgroups takes the other form: the same sums in the same order
    few = {k: v[:1].contiguous() for k, v in d.items()}
    again = out.t[:1].clone()
    all_ = out.t.clone()
    a = ops.delta_rule_step(**few, h=again)
    b = ops.delta_rule_step(**d, h=all_)
    assert torch.equal(again, all_[:1]) and torch.equal(a, b[:1])
