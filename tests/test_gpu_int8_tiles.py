"""Products of 8-bit rows in tiles of 128 x 128 and steps of 128, which ordinary
shapes like 2048 x 4096 x 4096 take, at sizes that end inside tiles and steps."""

import pytest
import torch

from gpu_util import Guarded
from quantized_recurrent_state_gdnq_amd import ops
from test_gpu_int8 import BF16, F32, near, random_codes
from gpu_util import DEV

pytestmark = pytest.mark.gpu

SIZES = [(2000, 4001, 144), (1990, 3500, 400), (2048, 4096, 16), (2047, 4095, 128), (1500, 4000, 1168)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product(M, N, K, dtype):
    a, sa = random_codes(M, K, M)
    w, sw = random_codes(N, K, N + 1)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(DEV) if (M + N) % 2 else None
    y = Guarded((M, N), dtype)
    ops.int8_matmul(a, sa, w, sw, bias, out_dtype=dtype, y=y.t)
    torch.cuda.synchronize()
    assert y.guards_intact()
    near(y.t, a, sa, w, sw, bias)


def test_largest_sums():
    """All codes -128: the largest sums that there are still fit."""
    M, N, K = 1990, 3500, 131056
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(N, device=DEV)
    y = ops.int8_matmul(a, one[:M], w, one, out_dtype=F32)
    assert (y == float(torch.tensor(K * 16384, dtype=torch.float32))).all()
