"""The ends of the number ranges in the 4-bit microscaled floats: every weight and the smallest
activations in the products that take activations as they are, blocks of subnormal numbers in the
encoder, and scales of rows that do not exist in every product."""
import numpy as np
import pytest
import torch

import w4a16_gemv_amd as amd
from tests.test_gpu_mxfp4 import BF, F32, FP, MAGNITUDES, TYPES, dev, encode, random_rows, same
from tests.test_gpu_mxfp4_contract import bits, padded

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def every_weight():
    """(Mxfp4Tensor, values fp64 [4096]): channel 16 E + c has the code c at element 39 with the scale E."""
    codes = torch.zeros(4096, 2, 16, dtype=torch.uint8)
    codes[:, 1, 3] = (torch.arange(4096) % 16 << 4).to(torch.uint8)
    scales = torch.full((4096, 2), 127, dtype=torch.uint8)
    scales[:, 1] = (torch.arange(4096) // 16).to(torch.uint8)
    m = torch.tensor(MAGNITUDES + [-v for v in MAGNITUDES], dtype=torch.float64)
    value = m[torch.arange(4096) % 16] * torch.exp2(torch.arange(4096).div(16, rounding_mode="floor").double() - 127)
    value[255 * 16:] = float("nan")
    return amd.Mxfp4Tensor.from_blocks(codes.to(dev()), scales.to(dev())), value


@pytest.mark.parametrize("xdtype", TYPES, ids=str)
@pytest.mark.parametrize("K", (64, 20000))
def test_gemv_every_weight(K, xdtype):
    """One activation, a power of two, and every value that a weight can have: the products are
    exact where fp32's normal numbers hold them.  Weights of 2^128 and more are infinities; an
    activation of fp16 or fp32 is a sum of parts, of which those of a power of two are zeros but
    for one, and an infinity times zero is NaN."""
    t, value = every_weight()
    if K > 64:       # rows that do not fit LDS
        c, s = t.blocks()
        blocks = -(-K // 32)
        codes = torch.zeros(4096, blocks, 16, dtype=torch.uint8, device=dev())
        scales = torch.full((4096, blocks), 127, dtype=torch.uint8, device=dev())
        codes[:, :2], scales[:, :2] = c, s
        t = amd.Mxfp4Tensor.from_blocks(codes, scales, K)
    value = torch.where(value.abs() >= 2.0 ** 128, value.sign() * INF, value).to(dev())
    powers = (0, -14, 14) if xdtype == FP else (0, -100, 100)
    x = torch.zeros(16, K, dtype=xdtype, device=dev())
    for i, p in enumerate(powers):
        x[i, 39] = 2.0 ** p
    y = amd.mxfp4_gemv(x, t, out_dtype=F32)
    for i, p in enumerate(powers):
        want = (value * 2.0 ** p).to(F32)
        if xdtype != BF:
            want[value.isinf()] = float("nan")
        # (sums among fp32's subnormal numbers may be zeros)
        small = (want.abs() < 2.0 ** -126) & (y[i] == 0)
        assert same(y[i][~small], want[~small]), f"2^{p}"
    assert same(y[3:], torch.where(value.isfinite(), 0.0, float("nan")).to(F32).expand(13, -1))


@pytest.mark.parametrize("xdtype", TYPES, ids=str)
def test_gemv_smallest_activations(xdtype):
    """Each subnormal number's bits times a large weight: down to 2^-133, as the header says."""
    lowest = {BF: -133, FP: -24, F32: -133}[xdtype]
    first = {BF: -126, FP: -14, F32: -126}[xdtype]
    codes = torch.zeros(8, 2, 16, dtype=torch.uint8, device=dev())
    codes[:, 1, 3] = 2 << 4          # 1.0
    power = 120
    t = amd.Mxfp4Tensor.from_blocks(codes, torch.full((8, 2), 127 + power, dtype=torch.uint8, device=dev()), 64)
    for e in range(lowest, first + 2):
        for odd in (1, 3, 5, 127):
            v = float(odd) * 2.0 ** e
            x = torch.zeros(16, 64, dtype=xdtype)
            x[:, 39] = torch.tensor(v, dtype=torch.float64).to(xdtype)
            got = amd.mxfp4_gemv(x.to(dev()), t, out_dtype=F32)
            assert same(got, (x[:, 39:40].double() * 2.0 ** power).to(F32).expand(16, 8)), (e, odd)


@pytest.mark.parametrize("dtype", (BF, F32), ids=str)
def test_quantize_subnormal_blocks(dtype):
    """Blocks around the smallest scale, 2^-127: largest magnitudes from 2^-133 to 2^-123, middles among the rest."""
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 7.0], dtype=torch.float64)
    rows = []
    for e in range(-127, -121):
        for top in range(e - 6, e + 1):
            v = torch.cat([ties, -ties, torch.tensor([0.0, 1.0], dtype=torch.float64)]) * 2.0 ** (top - 2)
            rows.append(v.to(dtype))
            if dtype == F32:
                moved = v.to(dtype)
                moved.view(torch.int32)[:-2] += 1
                rows.append(moved)
    x = torch.stack(rows)
    c, s = amd.mxfp4_quantize(x.to(dev())).blocks()
    codes, scales = encode(x)
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes)
    # and as the one-launch product encodes it: times ones of 2^120
    one = torch.full((4, 1, 16), 0x22, dtype=torch.uint8, device=dev())
    w = amd.Mxfp4Tensor.from_blocks(one, torch.full((4, 1), 247, dtype=torch.uint8, device=dev()))
    y = amd.mxfp4_linear(x[:16].to(dev()), w, out_dtype=F32)
    assert same(y, amd.mxfp4_gemm(amd.mxfp4_quantize(x[:16].to(dev())), w, out_dtype=F32))


# sizes of every kind of kernel, rows and channels off a tile of scales
SIZES = [(1, 70, 300), (13, 100, 4096), (17, 40, 129), (100, 20, 300), (333, 1007, 700), (700, 900, 1000), (2456, 3478, 256)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales_of_rows_past_the_last(M, N, K):
    """They may hold anything: no output of a product knows them."""
    x, xt = random_rows(1, M, K)
    w, wt = random_rows(2, N, K)
    a, b = (padded(t) if t.rows % 32 else t for t in (xt, wt))
    assert bits(amd.mxfp4_gemm(a, b, out_dtype=F32), amd.mxfp4_gemm(xt, wt, out_dtype=F32))
    for dtype in TYPES:
        v = torch.randn(M, K, device=dev()).to(dtype)
        assert bits(amd.mxfp4_linear(v, b, out_dtype=F32), amd.mxfp4_linear(v, wt, out_dtype=F32))
        if M <= 16:
            assert bits(amd.mxfp4_gemv(v, b, out_dtype=F32), amd.mxfp4_gemv(v, wt, out_dtype=F32))
    E = 3
    w, wt = random_rows(3, E * N, K)
    route = amd.moe_sort(torch.arange(M, device=dev()).view(M, 1) % E, E)
    a, b = (padded(t) if t.rows % 32 else t for t in (xt, wt))
    assert bits(amd.mxfp4_gemm_grouped(a, b, route, out_dtype=F32), amd.mxfp4_gemm_grouped(xt, wt, route, out_dtype=F32))
