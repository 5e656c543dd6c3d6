"""Microscaled 4-bit floating point (gdnq_mx_*) on the GPU: the codec bit for
bit against its definition, the product against exact sums in 64 bits.

Products of two codes with their powers of two are exact in fp32, so a sum of
K of them in fp32 in any order is off by at most K 2^-24 times the sum of
their magnitudes; a bf16 output adds half a step, 2^-8 of its value."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, Guarded, dev
from quantized_recurrent_state_gdnq_amd import _lib, ops

pytestmark = pytest.mark.gpu

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(x):
    """Definition, in float64: (codes 0..15 [..,K], scales [..,K/32])."""
    b = x.astype(np.float64).reshape(x.shape[:-1] + (-1, 32))
    top = np.abs(b).max(-1)
    s = np.where(top > 0, np.maximum(np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2, -127), -127).astype(int)
    m = np.abs(b) / 2.0 ** s[..., None]
    near = np.abs(m[..., None] - GRID)
    best = near.min(-1, keepdims=True)
    tie = near == best
    code = np.where(tie.sum(-1) == 1, tie.argmax(-1), 0)
    for i in (0, 2, 4, 6):  # of two equally near codes the even one
        code = np.where((tie.sum(-1) == 2) & tie[..., i], i, code)
    return (code + 8 * np.signbit(b)).reshape(x.shape), s + 127


def unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))


def decode(code, scales):
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(scales.shape + (32,)) * 2.0 ** (scales.astype(np.float64)[..., None] - 127)).reshape(code.shape)


def assert_codes(x, codes, scales, name=""):
    want, s = encode(x)
    got = unpack(codes.cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s, err_msg=name)
    zero = (want & 7) == 0  # the sign of a zero is not fixed
    assert ((got & 7)[zero] == 0).all(), name
    np.testing.assert_array_equal(got[~zero], want[~zero], err_msg=name)


def random_rows(rows, K, seed, dtype=torch.float32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=g)
    x *= torch.exp2(torch.round(torch.randn((rows, K // 32), generator=g) * spread)).repeat_interleave(32, 1)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (7, 96), (64, 1056), (513, 4096)])
def test_codec(rows, K, dtype):
    x = random_rows(rows, K, rows + K, dtype)
    c, s = Guarded((rows, K // 2), torch.uint8, 77), Guarded((rows, K // 32), torch.uint8, 77)
    ops.mx_quantize(x.to(DEV), c.t, s.t)
    assert c.guards_intact() and s.guards_intact()
    assert_codes(x.double().numpy(), c.t, s.t)


def test_codec_every_mantissa_and_tie():
    """Every bf16 value of two binades against block maxima of all mantissas:
    every rounding border, from below, on it and above."""
    m = torch.arange(0, 1 << 15, dtype=torch.int32)
    x = (m << 16).view(torch.float32)
    x = x[torch.isfinite(x)]
    near = x[(x > 2.0 ** -6) & (x < 8.0)]
    x = torch.zeros(near.numel(), 32)
    x[:, 0] = 7.5
    x[:, 1], x[:, 2] = near, -near
    x[:, 3] = torch.nextafter(near, torch.tensor(9.0))
    x[:, 4] = torch.nextafter(near, torch.tensor(0.0))
    assert_codes(x.double().numpy(), *ops.mx_quantize(x.to(DEV)))
    xb = x.bfloat16()
    assert_codes(xb.double().numpy(), *ops.mx_quantize(xb.to(DEV)))


def test_codec_of_more_values_than_one_launch_takes():
    """2^34 values are a launch; the rows on both sides of its end against the
    same rows alone."""
    rows, K = 2 ** 14 + 8, 2 ** 20
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of free device memory")
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    some = [0, 1, 2 ** 14 - 2, 2 ** 14 - 1, 2 ** 14, 2 ** 14 + 1, rows - 1]
    g = torch.Generator(device=DEV).manual_seed(5)
    part = torch.randn(len(some), K, generator=g, device=DEV).bfloat16()
    x[some] = part
    codes = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, K // 32), 0xEE, dtype=torch.uint8, device=DEV)
    ops.mx_quantize(x, codes, scales)
    del x
    want_codes, want_scales = ops.mx_quantize(part)
    assert torch.equal(codes[some], want_codes) and torch.equal(scales[some], want_scales)
    for r in (2, 2 ** 13, 2 ** 14 - 3, 2 ** 14 + 2, rows - 2):
        assert not codes[r].any() and not scales[r].any()
    del codes, scales
    torch.cuda.empty_cache()


def test_codec_extremes():
    tiny = 2.0 ** -149
    rows = [[0.0] * 32, [tiny] * 32, [2.0 ** -126] + [2.0 ** -128] * 31, [2.0 ** -125] + [tiny] * 31,
            [3.4028234e38] + [1e38] * 31, [2.0 ** -120, -(2.0 ** -122)] * 16, [-0.0] * 31 + [1.0]]
    x = torch.tensor(rows, dtype=torch.float32)
    assert_codes(x.double().numpy(), *ops.mx_quantize(x.to(DEV)))


def test_codec_and_product_of_nan_and_infinity():
    """Such a block has the NaN scale, and only its own rows' results are NaN."""
    x, w = random_rows(40, 256, 1), random_rows(24, 256, 2)
    x[3, 40], x[17, 200] = float("nan"), float("inf")
    codes, scales = ops.mx_quantize(x.to(DEV))
    s = scales.cpu().numpy()
    assert s[3, 1] == 255 and s[17, 6] == 255 and (s == 255).sum() == 2
    wc, ws = ops.mx_quantize(w.to(DEV))
    y = ops.mx_matmul(codes, scales, wc, ws, out_dtype=torch.float32).cpu()
    bad = torch.zeros(40, dtype=torch.bool)
    bad[3] = bad[17] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def check_product(x, w, out_dtype):
    rows, cols, K = x.shape[0], w.shape[0], x.shape[1]
    ac, asc = ops.mx_quantize(x.to(DEV))
    wc, wsc = ops.mx_quantize(w.to(DEV))
    out = Guarded((rows, cols), out_dtype)
    ops.mx_matmul(ac, asc, wc, wsc, out_dtype=out_dtype, y=out.t)
    assert out.guards_intact()
    a = decode(unpack(ac.cpu().numpy()), asc.cpu().numpy())
    b = decode(unpack(wc.cpu().numpy()), wsc.cpu().numpy())
    want = a @ b.T
    tol = K * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T) + 1e-37
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(out.t.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.2f} of the bound, {np.sum(err > tol)} off"
    y = ops.mx_linear(x.to(DEV), wc, wsc, out_dtype=out_dtype)
    assert torch.equal(y, out.t)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,K", [(1, 1, 32), (1, 16, 128), (2, 17, 160), (5, 100, 512), (16, 64, 2048), (17, 130, 1056),
                                         (33, 333, 544), (64, 512, 4096), (65, 257, 768), (127, 129, 96), (128, 128, 128),
                                         (129, 255, 480), (300, 515, 2080), (513, 260, 1024), (1000, 1111, 992)])
def test_product(rows, cols, K, out_dtype):
    check_product(random_rows(rows, K, rows, torch.bfloat16), random_rows(cols, K, cols + 1), out_dtype)


@pytest.mark.parametrize("rows", [1, 3, 8, 15, 16, 24, 31, 32, 40, 48, 63, 96, 100, 160, 200, 256, 257])
def test_product_rows(rows):
    check_product(random_rows(rows, 1088, rows, torch.bfloat16), random_rows(144, 1088, 7), torch.bfloat16)


@pytest.mark.parametrize("K", [32 * k for k in (1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 31, 33, 63, 65)])
@pytest.mark.parametrize("rows", [20, 300])
def test_product_depths(K, rows):
    check_product(random_rows(rows, K, rows, torch.bfloat16), random_rows(272, K, 7), torch.float32)


# sizes of the larger tiles: 128 x 128 (two on a CU), 256 x 256, each with whole and ragged steps and edges
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,K", [(2049, 2301, 32), (2304, 2176, 1024), (2049, 2301, 1312), (3585, 3331, 32),
                                         (3329, 3584, 288), (3584, 3584, 512), (3500, 3333, 992), (3585, 3600, 1280)])
def test_product_large_tiles(rows, cols, K, out_dtype):
    check_product(random_rows(rows, K, rows, torch.bfloat16), random_rows(cols, K, cols + 1), out_dtype)


def test_scales_pair_with_their_blocks():
    """One nonzero block at a time, every power of two its own: a scale taken
    from a neighbour, or a block multiplied by another, is a wrong power."""
    K, blocks = 1024, 32
    x, w = torch.zeros(blocks + 300, K), torch.zeros(blocks + 20, K)
    for i in range(blocks):
        x[i, 32 * i:32 * i + 32] = 2.0 ** (i - 10)
        w[i, 32 * i:32 * i + 32] = 2.0 ** (3 - i)
    wc, ws = ops.mx_quantize(w.to(DEV))
    for rows in (blocks, blocks + 300):
        y = ops.mx_linear(x[:rows].to(DEV), wc, ws).cpu()
        want = torch.zeros(rows, blocks + 20)
        for i in range(blocks):
            want[i, i] = 32 * 2.0 ** -7
        assert torch.equal(y, want)


def test_leading_dimensions_streams_and_graph():
    x = random_rows(6 * 50, 512, 3, torch.bfloat16).view(6, 50, 512).to(DEV)
    wc, ws = ops.mx_quantize(random_rows(200, 512, 4).to(DEV))
    flat = ops.mx_linear(x.view(300, 512), wc, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = ops.mx_linear(x, wc, ws)
        few = ops.mx_linear(x[0, :3].contiguous(), wc, ws)
    torch.cuda.synchronize()
    assert torch.equal(side.view(300, 200), flat)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = ops.mx_linear(x, wc, ws), ops.mx_linear(x[0, :3].contiguous(), wc, ws)
    for seed in range(3):
        if seed:
            x.copy_(random_rows(300, 512, 30 + seed, torch.bfloat16).view(6, 50, 512))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), z.clone()
        want = ops.mx_linear(x, wc, ws), ops.mx_linear(x[0, :3].contiguous(), wc, ws)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert few.shape == (3, 200)


def test_empty():
    wc, ws = ops.mx_quantize(torch.zeros(8, 64, device=DEV))
    assert ops.mx_linear(torch.zeros(0, 64, device=DEV), wc, ws).shape == (0, 8)
    assert ops.mx_quantize(torch.zeros(0, 64, device=DEV))[0].shape == (0, 32)


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    wc, ws = ops.mx_quantize(torch.zeros(8, 64, device=DEV))
    for bad in (x[:, :40].contiguous(), x.half(), x.cpu(), torch.zeros(64, 4, device=DEV).t()):
        with pytest.raises(ValueError):
            ops.mx_quantize(bad)
    for args in ((x, wc[:, :16].contiguous(), ws), (x, wc, ws[:4]), (x, wc.char(), ws), (x[:, :32].contiguous(), wc, ws)):
        with pytest.raises(ValueError):
            ops.mx_linear(*args)
    with pytest.raises(ValueError):
        ops.mx_linear(x, wc, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ops.mx_linear(x, wc, ws, y=torch.zeros(4, 9, device=DEV))
    with pytest.raises(_lib.GdnqError, match="WORKSPACE"):
        ops.mx_linear(x, wc, ws, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(_lib.GdnqError, match="ALIAS"):
        codes = torch.zeros(8, 64, device=DEV)
        ops.mx_quantize(codes, codes.view(torch.uint8).view(-1)[:256].view(8, 32))


@pytest.mark.parametrize("rows", [1, 2, 9, 16])
@pytest.mark.parametrize("cols,K", [(4096, 544), (4112, 544), (4097, 1056), (8192, 1024), (8193, 1056), (8208, 992), (33000, 96)])
def test_few_rows_many_columns(rows, cols, K):
    """On both sides of the numbers of columns at which the kernel changes;
    fp32 results show the order of the sums, which is the same in both calls."""
    check_product(random_rows(rows, K, rows, torch.bfloat16), random_rows(cols, K, cols + 1), torch.float32)


def test_product_allocates_its_result_alone():
    ac, asc = ops.mx_quantize(torch.zeros(2048, 4096, device=DEV))
    wc, wsc = ops.mx_quantize(torch.zeros(64, 4096, device=DEV))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y = ops.mx_matmul(ac, asc, wc, wsc)
    assert torch.cuda.max_memory_allocated() - before == y.numel() * 2  # 256 KiB; the rows' codes are 4 MiB
    given = torch.empty(64, dtype=torch.uint8, device=DEV)  # one that is given is not used, whatever its size
    assert torch.equal(ops.mx_matmul(ac, asc, wc, wsc, workspace=given), y)
