"""8-bit rows and their product (gdnq_int_*) on the GPU: the codes against the
codec's definition in the library's oracle, exactly, and the product against whole
numbers in 64 bits: a sum of whole numbers is exact, its conversion, two scales
and the bias are four roundings of 2^-24 (of the terms' magnitudes), and a bf16
result adds half a step, 2^-8."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded
import oracle
from quantized_recurrent_state_gdnq_amd import _lib, ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32


def codes_of(x):
    x = x.float().cpu().numpy()
    c, s = oracle.quantize_rows(x)
    return torch.from_numpy(np.asarray(c)), torch.from_numpy(np.asarray(s))


def near(got, a, sa, w, sw, bias):
    whole = (a.double().cpu() @ w.double().cpu().t())
    scaled = whole * sa.double().cpu()[:, None] * sw.double().cpu()
    want = scaled if bias is None else scaled + bias.double().cpu()
    err = (got.double().cpu() - want).abs()
    size = scaled.abs() + (0 if bias is None else bias.double().cpu().abs())
    allowed = (4 * U) * size + HALF[got.dtype] * (want.abs() + 4 * U * size) + 1e-38
    assert (err <= allowed).all(), float((err / allowed).max())


def random_codes(rows, depth, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-127, 128, (rows, depth), generator=g, dtype=torch.int8).to(DEV),
            (torch.rand(rows, generator=g) + 0.5).to(DEV) / 127)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,depth", [(1, 16), (7, 48), (3, 512), (5, 528), (4, 2048), (9, 2064), (2, 4096), (3, 4112),
                                        (2, 8192), (2, 8208), (1, 131056), (300, 64)])
def test_codes(rows, depth, dtype):
    g = torch.Generator().manual_seed(rows + depth)
    x = torch.randn((rows, depth), generator=g).to(dtype)
    x[0, 5] = 9.0
    want_c, want_s = codes_of(x)
    c, s = ops.int8_quantize(x.to(DEV))
    assert torch.equal(s.cpu(), want_s) and torch.equal(c.cpu(), want_c)


def test_codes_at_ties_zeros_and_tiny_rows():
    x = torch.zeros((6, 32))
    x[0] = torch.arange(32) - 15.5          # halves: scale 127 / 127 = 1 with the next line
    x[0, 0] = 127.0
    x[2, 3] = 1e-44                          # a scale that rounds to 0
    x[3] = torch.linspace(-1e-38, 1e-38, 32)  # a subnormal scale
    x[4] = 3e38 * torch.linspace(-1, 1, 32)
    x[5] = -0.0
    want_c, want_s = codes_of(x)
    c, s = ops.int8_quantize(x.to(DEV))
    assert torch.equal(s.cpu(), want_s) and torch.equal(c.cpu(), want_c)


def test_rows_that_are_not_finite():
    """Scale NaN, codes 0, and only that row's results are NaN."""
    for depth in (64, 1024, 9008):
        x = torch.randn((4, depth)).to(DEV)
        clean = ops.int8_quantize(x)
        x[1, depth - 1], x[2, 0] = float("nan"), float("-inf")
        c, s = ops.int8_quantize(x)
        assert torch.isnan(s[1:3]).all() and (c[1:3] == 0).all()
        assert torch.equal(c[[0, 3]], clean[0][[0, 3]]) and torch.equal(s[[0, 3]], clean[1][[0, 3]])
        w, sw = random_codes(5, depth, 1)
        y = ops.int8_linear(x, w, sw)
        assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3]]).all()


# every kernel, with sizes that end inside its tiles
SIZES = [(1, 1, 16), (1, 16, 64), (16, 100, 80), (3, 4099, 272), (17, 33, 1040), (33, 7000, 96), (64, 4096, 512),
         (100, 130, 4096), (65, 65, 16), (129, 1000, 528), (700, 800, 272), (1001, 1111, 2064), (513, 6000, 144),
         (2049, 6200, 80), (4000, 4001, 400), (300, 40000, 16)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product(M, N, K, dtype):
    a, sa = random_codes(M, K, M)
    w, sw = random_codes(N, K, N + 1)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(DEV) if (M + N) % 2 else None
    near(ops.int8_matmul(a, sa, w, sw, bias, out_dtype=dtype), a, sa, w, sw, bias)


def test_largest_sums():
    """All codes -128: the largest sums that there are still fit."""
    K = 131056
    for M, N in ((2, 20), (70, 70), (200, 520)):
        a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
        w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
        one = torch.ones(max(M, N), device=DEV)
        y = ops.int8_matmul(a, one[:M], w, one[:N], out_dtype=F32)
        assert (y == float(np.float32(K * 16384))).all()


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (16, 4096, 1024), (64, 512, 4096), (333, 257, 2080), (3, 8, 9008)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear(M, N, K, dtype):
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, K), generator=g).to(dtype).to(DEV)
    w, sw = ops.int8_quantize(torch.randn((N, K), generator=g).to(DEV) / K ** 0.5)
    bias = torch.randn(N, generator=g).to(DEV)
    c, s = ops.int8_quantize(x)
    for b in (None, bias):
        y = ops.int8_linear(x, w, sw, b)
        assert y.dtype == dtype
        near(y, c, s, w, sw, b)
        assert torch.equal(y, ops.int8_matmul(c, s, w, sw, b, out_dtype=dtype))
    y = ops.int8_linear(x.view(1, M, K), w, sw, out_dtype=F32)
    assert y.shape == (1, M, N) and y.dtype == F32


def test_writes_stay_inside():
    for M, N, K in ((5, 37, 48), (70, 129, 272), (1001, 1111, 80)):
        a, sa = random_codes(M, K, 1)
        w, sw = random_codes(N, K, 2)
        for dtype in (BF16, F32):
            y = Guarded((M, N), dtype)
            ops.int8_matmul(a, sa, w, sw, out_dtype=dtype, y=y.t)
            torch.cuda.synchronize()
            assert y.guards_intact() and torch.isfinite(y.t).all()
        c, s = Guarded((M, K), torch.int8), Guarded((M,), F32)
        ops.int8_quantize(torch.randn(M, K, device=DEV), c.t, s.t)
        torch.cuda.synchronize()
        assert c.guards_intact() and s.guards_intact()


def test_graph_replays():
    x = torch.randn(64, 1024, device=DEV, dtype=BF16)
    w, sw = ops.int8_quantize(torch.randn(512, 1024, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.int8_linear(x, w, sw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.int8_linear(x, w, sw)
    for i in range(4):
        x.copy_(torch.randn(64, 1024, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want = ops.int8_linear(x, w, sw)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_two_streams_at_once():
    w, sw = random_codes(1000, 2048, 1)
    xs = [torch.randn(300, 2048, generator=torch.Generator().manual_seed(s)).to(DEV) for s in (1, 2)]
    want = [ops.int8_linear(x, w, sw) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(ops.int8_linear(xs[i], w, sw))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def test_empty_and_refusals():
    w, sw = random_codes(8, 32, 1)
    x = torch.randn(3, 32, device=DEV)
    assert ops.int8_linear(x[:0], w, sw).shape == (0, 8)
    assert ops.int8_quantize(x[:0])[0].shape == (0, 32)
    bad = [lambda: ops.int8_quantize(x[:, :20].contiguous()), lambda: ops.int8_quantize(x.half()),
           lambda: ops.int8_linear(x, w[:, :16].contiguous(), sw), lambda: ops.int8_linear(x, w, sw[:3]),
           lambda: ops.int8_linear(x, w.to(torch.uint8), sw), lambda: ops.int8_linear(x, w, sw, bias=sw[:2]),
           lambda: ops.int8_linear(x.t(), w, sw), lambda: ops.int8_linear(x, w, sw, out_dtype=torch.float16),
           lambda: ops.int8_matmul(w[:3], sw[:2], w, sw), lambda: ops.int8_linear(x, w, sw, y=x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(_lib.GdnqError, match="SHAPE"):
        ops.int8_matmul(torch.zeros(1, 24, dtype=torch.int8, device=DEV), sw[:1], torch.zeros(8, 24, dtype=torch.int8, device=DEV), sw)
    with pytest.raises(_lib.GdnqError, match="WORKSPACE"):
        ops.int8_linear(x, w, sw, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
