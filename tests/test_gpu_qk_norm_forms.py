"""Forms of the norm of queries and keys that its other tests' sizes do not reach:
no rotation, in rows of whole 16-byte pieces and in others, and all columns of a
row of 256 turned, whose halves lie in two halves of a team of 32 lanes."""

import pytest

from test_gpu_qk_norm import BF16, F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,Hq,Hk,D,r", [(6, 2, 1, 128, 0), (5, 3, 1, 64, 0), (3, 2, 2, 256, 0), (3, 1, 1, 90, 0), (4, 2, 1, 512, 0),
                                         (700, 3, 2, 128, 0), (4, 2, 1, 256, 256), (900, 2, 1, 256, 256), (3, 1, 2, 512, 512)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
def test_forms(N, Hq, Hk, D, r, dtype, fused):
    d, more = make(N, Hq, Hk, D, r, dtype, True, 5000, seed=D + r, fused=fused)
    check(d, more)
    check(d, more, norm="l2", eps=1e-5)
    if r:
        check(d, more, interleaved=True)
