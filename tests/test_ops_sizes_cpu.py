"""Sizes beyond 32 bits are refused by the wrappers of the scan, the group norm
and the microscaled product: the C parameters hold 32 bits, and a call must not
go on with the low ones of a larger size.  Tensors without memory stand in for
the large ones (a bf16 tensor of 2^32 + 10 values, 8 GiB, is no large one on
the device)."""

import pytest
import torch

from quantized_recurrent_state_gdnq_amd import ops

BIG = 2 ** 32 + 10


@pytest.fixture
def meta(monkeypatch):
    """Tensors of the given shape on no device, that pass for GPU tensors."""
    monkeypatch.setattr(ops, "_need", lambda t, *a, **k: t)

    def make(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")
    return make


@pytest.mark.parametrize("shape", [(1, BIG, 1), (BIG, 1, 1), (1, 1, BIG)])
def test_scan(meta, shape):
    x = meta(*shape)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.gated_scan(x, x)
    carry = meta(-(-shape[0] * shape[1] // 128), shape[2], dtype=torch.float32)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.gated_scan_backward(x, x, x, carry)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.scan_workspace_size(x)


def test_packed_scan_and_step(meta):
    x, cu = meta(BIG, 1), meta(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.gated_scan(x, x, cu_seqlens=cu)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.scan_workspace_size(x, cu)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.gated_scan_step(x, x, meta(BIG, 1, dtype=torch.float32))


@pytest.mark.parametrize("shape", [(BIG, 1, 8), (3, BIG // 3, 1, 8), (1, BIG, 8), (1, 1, BIG)])
def test_norm(meta, shape):
    x = meta(*shape)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.group_norm(x)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.group_norm_backward(x, x)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.group_norm_workspace_size(x)


def test_product(meta):
    u8 = torch.uint8
    few, many = (meta(4, 16, dtype=u8), meta(4, 1, dtype=u8)), (meta(BIG, 16, dtype=u8), meta(BIG, 1, dtype=u8))
    for a, w in ((few, many), (many, few)):
        with pytest.raises(ValueError, match="2\\^31"):
            ops.mx_matmul(*a, *w)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.mx_linear(meta(4, 32), *many)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.mx_linear(meta(2, BIG // 2, 32), *few)
    deep = 2 ** 32 + 64
    with pytest.raises(ValueError, match="2\\^31"):
        ops.mx_quantize(meta(1, deep))
    with pytest.raises(ValueError, match="2\\^31"):
        ops.mx_linear(meta(1, deep), meta(1, deep // 2, dtype=u8), meta(1, deep // 32, dtype=u8))
    with pytest.raises(ValueError, match="2\\^31"):
        ops.mx_workspace_size(4, BIG, 32)


def test_largest_sizes_pass():
    ops._sizes(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)
    assert ops.mx_workspace_size(1, 16, 32) > 0
