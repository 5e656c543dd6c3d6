"""The plain form of the 8-bit linear layer's codec in perf/more_operators.py on
the GPU: its scales and codes are the oracle's bit for bit, as the library's
kernels' are, so that the two can be compared."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import DEV
import oracle

pytestmark = pytest.mark.gpu


def plain():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators_cases", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_plain_codes(dtype):
    """The 127th of a maximum is a division, rounded once: the product with the
    reciprocal of 127 is another value for one row in twenty."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn((4096, 64), generator=g).to(dtype)
    codes, scales = plain()._codes(x.to(DEV))
    want_codes, want_scales = oracle.quantize_rows(x.float().numpy())
    assert torch.equal(scales.cpu(), torch.from_numpy(np.asarray(want_scales)))
    assert torch.equal(codes.cpu(), torch.from_numpy(np.asarray(want_codes)))
