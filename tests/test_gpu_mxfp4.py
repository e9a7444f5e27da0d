"""GPU parity of the 4-bit microscaled floats (include/mxfp4.h) against the
definitions in 64 bits.

The encoder is exact: codes and scales are compared as they are.  The products of two
values are exact, and where a sum of magnitudes, counted in the smallest unit that any
product has, stays below 2^24, so is every partial sum in any order: then outputs are
compared bit for bit with the exact sum rounded once (`exactly`).  Elsewhere a sum of K
products is within terms * 2^-23 * S of the exact one, S the sum of the magnitudes and
terms the additions that follow one another (each rounds by 2^-24 of its result at
most, which is no larger than S, and a matrix instruction's own sum by as much again),
and the output's rounding adds half a step of the type."""
import ctypes as C

import numpy as np
import pytest
import torch

import w4a16_gemv_amd as amd

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF, FP, F32]
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def dev():
    return torch.device("cuda:0")


def plan(M, N, K, E=0, room=1 << 62):
    """The kernel that a product goes to (needs no GPU)."""
    a, b = C.c_int32(), C.c_int32()
    assert amd.load().nf4_probe_mxfp4_plan(M, N, K, E, room, C.byref(a), C.byref(b)) == 0
    return a.value, b.value


def same(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Equal bit for bit, any NaN equal to any other and 0 to -0."""
    a, b = a.cpu(), b.cpu()
    return a.dtype == b.dtype and a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def decode(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """fp64 [rows][K] of codes [rows][blocks][16] and scales [rows][blocks]."""
    table = np.array(MAGNITUDES + [-m for m in MAGNITUDES])
    v = np.stack([table[codes & 15], table[codes >> 4]], -1).reshape(*scales.shape, 32)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(scales.shape[0], -1)[:, :K]


def encode(x: torch.Tensor):
    """(codes [rows][blocks][16], scales [rows][blocks]) of a CPU tensor's rows, by definition."""
    v = x.double().numpy()
    rows, K = v.shape
    blocks = -(-K // 32)
    full = np.zeros((rows, blocks * 32))
    full[:, :K] = v
    full = full.reshape(rows, blocks, 32)
    finite = np.isfinite(full).all(2)
    full = np.where(finite[..., None], full, 0.0)
    peak = np.abs(full).max(2)
    power = np.where(peak > 0, np.frexp(peak)[1] - 1 - 2, -127)
    e = np.maximum(power, -127)
    t = np.abs(full) * np.exp2(-e.astype(np.float64))[..., None]
    code = np.zeros(t.shape, np.uint8)
    # between the magnitudes i and i + 1: past the middle, and on it where i is odd
    for i in range(7):
        middle = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        code += ((t > middle) | ((t == middle) & (i % 2 == 1))).astype(np.uint8)
    code |= np.signbit(full).astype(np.uint8) << 3
    code[~finite] = 0
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scales


def random_rows(seed, rows, K, low=126, high=129):
    """(values fp64 on the GPU, Mxfp4Tensor) of random codes with scales from low to high - 1."""
    rng = np.random.default_rng(seed)
    blocks = -(-K // 32)
    codes = rng.integers(0, 256, (rows, blocks, 16), dtype=np.uint8)
    scales = rng.integers(low, high, (rows, blocks)).astype(np.uint8)
    t = amd.Mxfp4Tensor.from_blocks(torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev()), K)
    return torch.from_numpy(decode(codes, scales, K)).to(dev()), t


def exactly(x, w, unit, dtype):
    """x w^T rounded once, after checking that no partial sum can round: all products are
    multiples of unit, and their magnitudes add up to less than 2^24 of them."""
    assert float((x.abs() @ w.abs().t()).max()) / unit < 2 ** 24
    return (x @ w.t()).to(F32).to(dtype)


GUARD = 96


def guarded(rows, N, dtype):
    """(whole buffer, view [rows][N] inside it); the rest holds a pattern."""
    whole = torch.full((rows * N + 2 * GUARD,), 7.25, dtype=dtype, device=dev())
    return whole, whole[GUARD:GUARD + rows * N].view(rows, N)


def untouched(whole, n):
    return bool((whole[:GUARD] == 7.25).all()) and bool((whole[GUARD + n:] == 7.25).all())


# --- the encoder -------------------------------------------------------------

QUANT = [(1, 1), (1, 7), (3, 8), (2, 31), (5, 32), (4, 33), (1, 4096), (7, 127), (9, 128), (3, 129), (2, 255), (33, 257),
         (6, 511), (3, 4099), (2, 8193), (65, 100), (300, 33), (1, 40001), (1030, 128), (2050, 70), (31, 1501)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,K", QUANT)
def test_quantize(rows, K, dtype):
    g = torch.Generator().manual_seed(rows * 1000 + K)
    x = (torch.randn(rows, K, generator=g) * torch.rand(rows, 1, generator=g) * 5).to(dtype)
    x[0, K // 2] = 0.0
    codes, scales = encode(x)
    # a row base that is aligned to nothing but the element
    room = torch.zeros(rows * K + 1, dtype=dtype, device=dev())
    for shift in (0, 1):
        view = room[shift:shift + rows * K].view(rows, K)
        view.copy_(x)
        t = amd.mxfp4_quantize(view)
        c, s = t.blocks()
        assert np.array_equal(s.cpu().numpy(), scales), "scales differ"
        assert np.array_equal(c.cpu().numpy(), codes), "codes differ"
        assert not t.data[:, codes.shape[1] * 16:].any(), "codes past the last block"
        for out in TYPES:
            assert same(t.dequant(out_dtype=out), torch.from_numpy(decode(codes, scales, K)).to(F32).to(out))


def test_scale_layout():
    """The bytes lie where the format says, with zeros past a row's last block."""
    rows, K = 70, 1501
    x = torch.randn(rows, K, generator=torch.Generator().manual_seed(1)) * torch.rand(rows, 1) * 100
    _, scales = encode(x)
    t = amd.mxfp4_quantize(x.to(dev()), out=amd.Mxfp4Tensor(
        torch.full((rows, 768), 255, dtype=torch.uint8, device=dev()),
        torch.full((3 * 6 * 256,), 255, dtype=torch.uint8, device=dev()), K))
    flat = t.scale.cpu().numpy()
    for r in range(rows):
        for b in range(48):
            byte = flat[((r // 32) * 6 + b // 8) * 256 + (b // 4 % 2) * 128 + (r % 32) * 4 + b % 4]
            assert byte == (scales[r, b] if b < 47 else 0), (r, b)
    # rows past the last are left alone
    assert (flat.reshape(3, 6, 2, 32, 4)[2, :, :, 6:] == 255).all()
    back = amd.Mxfp4Tensor.from_blocks(*t.blocks(), K)
    assert torch.equal(back.data, t.data) and torch.equal(back.dequant(out_dtype=F32), t.dequant(out_dtype=F32))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_rounding_borders(dtype):
    """Values on and next to the middles between magnitudes, of every sign and scale that the type has."""
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 7.0], dtype=torch.float64)
    lo, hi = {BF: (-120, 120), FP: (-12, 12), F32: (-126, 125)}[dtype]
    rows = []
    for e in range(lo, hi + 1, 3):
        for move in (0, 1, -1):
            v = (torch.cat([ties, -ties, torch.tensor([4.0], dtype=torch.float64)]) * 2.0 ** e).to(dtype)
            bits = v.view(torch.int32 if dtype == F32 else torch.int16)
            bits[:-1] += move
            rows.append(v)
    x = torch.stack(rows)
    c, s = amd.mxfp4_quantize(x.to(dev())).blocks()
    codes, scales = encode(x)
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_extremes(dtype):
    """Blocks of zeros, of the smallest and the largest numbers, and blocks that are not finite."""
    info = torch.finfo(dtype)
    x = torch.zeros(12, 96, dtype=dtype)
    x[1, :40] = -0.0
    x[2, 5], x[2, 70] = info.smallest_normal, -info.smallest_normal
    x[3] = info.max
    x[4, ::2] = info.min
    x[5, 3], x[5, 64] = float("nan"), 1.0
    x[6, 33], x[6, 2] = float("inf"), 3.0
    x[7, 95], x[7, 94] = float("-inf"), float("nan")
    tiny = torch.ones(2, dtype=torch.int32 if dtype == F32 else torch.int16).view(dtype)[0]
    x[8, 7], x[8, 40] = tiny, -tiny
    x[9] = info.smallest_normal
    x[9, 1::3] = tiny
    x[10, :32] = info.max
    x[10, 5] = tiny
    t = amd.mxfp4_quantize(x.to(dev()))
    codes, scales = encode(x)
    c, s = t.blocks()
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes)
    for out in TYPES:
        assert same(t.dequant(out_dtype=out), torch.from_numpy(decode(codes, scales, 96)).to(F32).to(out))


def test_every_code_and_scale_decodes():
    """All 256 scales (255 is NaN, and what passes a type's range is an infinity) with all codes."""
    codes = torch.arange(256, dtype=torch.uint8).view(16, 16)[None].repeat(256, 1, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    t = amd.Mxfp4Tensor.from_blocks(codes.to(dev()), scales.to(dev()))
    want = torch.from_numpy(decode(codes.numpy(), scales.numpy(), 512))
    for out in TYPES:
        # (to fp32 first: exact, or an infinity)
        assert same(t.dequant(out_dtype=out), want.to(F32).to(out))


def test_from_blocks_cuts_what_lies_past_K():
    for K in (33, 40, 63):
        codes = torch.full((3, 2, 16), 0x77, dtype=torch.uint8, device=dev())
        t = amd.Mxfp4Tensor.from_blocks(codes, torch.full((3, 2), 127, dtype=torch.uint8, device=dev()), K)
        assert (t.dequant() == 6).all() and t.dequant().shape == (3, K)
        whole = torch.stack([t.data & 15, t.data >> 4], -1).view(3, -1)
        assert (whole[:, :K] == 7).all() and not whole[:, K:].any()


def test_quantize_flattens_and_strides_are_refused():
    x = torch.randn(2, 3, 70, device=dev())
    t = amd.mxfp4_quantize(x)
    assert (t.rows, t.K) == (6, 70) and torch.equal(t.data, amd.mxfp4_quantize(x.view(6, 70)).data)
    with pytest.raises(ValueError, match="contiguous"):
        amd.mxfp4_quantize(x.transpose(0, 1))
    assert amd.mxfp4_quantize(torch.zeros(0, 64, device=dev())).dequant().shape == (0, 64)
    assert amd.mxfp4_quantize(torch.zeros(4, 0, device=dev())).dequant().shape == (4, 0)


# --- the products ------------------------------------------------------------

DENSE = [(1, 1, 1), (1, 8, 18), (3, 17, 33), (16, 100, 129), (15, 33, 255), (1, 4099, 1501), (1, 8, 4175), (2, 100, 9999),
         (1, 9, 12576), (4, 40, 20000), (16, 65, 12000), (17, 40, 128), (100, 20, 300), (42, 2766, 16), (1, 8, 22885),
         (3, 627, 20100), (1271, 8, 15833), (1172, 197, 8691), (165, 476, 34494), (2210, 490, 17), (65, 2759, 43069),
         (1962, 257, 16), (4148, 195, 3334), (5441, 520, 538), (69, 3280, 53757), (3415, 4261, 267), (1996, 2597, 2779),
         (333, 4099, 1501), (5077, 4142, 515), (1750, 2128, 519), (3722, 4596, 524), (300, 300, 300), (130, 129, 1000),
         (3, 16400, 2000), (5, 65600, 500)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_gemm(M, N, K):
    """Every kernel and split, with and without a workspace; nothing outside y is written."""
    # scales 2^0 and 2^1: products are multiples of 1/4; for long rows all one scale
    x, xt = random_rows(M + K, M, K, 127, 129 if K < 10000 else 128)
    w, wt = random_rows(N + 7 * K, N, K, 127, 129 if K < 10000 else 128)
    for dtype in TYPES:
        want = exactly(x, w, 0.25, dtype)
        whole, y = guarded(M, N, dtype)
        amd.mxfp4_gemm(xt, wt, y=y)
        assert same(y, want), f"{dtype}"
        assert untouched(whole, M * N)
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    assert same(amd.mxfp4_gemm(xt, wt, out_dtype=F32, workspace=none), exactly(x, w, 0.25, F32))


LINEAR = [(1, 4096, 4096), (2, 33, 7), (13, 1100, 1024), (16, 40, 9999), (1, 70, 20000), (17, 64, 300), (40, 100, 129),
          (333, 411, 1501), (700, 900, 160), (1, 40, 9999), (2, 70, 6001), (3, 16400, 2000), (2, 32800, 1000), (5, 65600, 500)]


@pytest.mark.parametrize("xdtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(M, N, K, xdtype):
    """Against the codes' exact products where no sum can round, and for any
    activations; a vector gives a vector."""
    x, _ = random_rows(M + K, M, K, 127, 129 if K < 10000 else 128)
    w, wt = random_rows(N, N, K, 127, 129 if K < 10000 else 128)
    room = torch.empty(M * K + 1, dtype=xdtype, device=dev())
    g = torch.Generator(device=dev()).manual_seed(M + K)
    noise = torch.randn(M, K, generator=g, device=dev())
    coded = amd.mxfp4_quantize(noise.to(xdtype)).dequant(out_dtype=F32).double()
    want = coded @ w.t()
    for shift in (0, 1):
        to = room[shift:shift + M * K].view(M, K)
        for dtype in TYPES:
            to.copy_(x)  # (every value of a code fits the types, and its block gets the same values again)
            whole, y = guarded(M, N, dtype)
            assert amd.mxfp4_linear(to, wt, y=y) is y
            assert same(y, exactly(x, w, 0.25, dtype)) and untouched(whole, M * N)
            to.copy_(noise)
            got = amd.mxfp4_linear(to, wt, out_dtype=dtype).double()
            assert ((got - want).abs() <= bound(coded, w, want, K / 64 + 17, dtype)).all()
    if M == 1:
        y = torch.empty(N, dtype=F32, device=dev())
        assert amd.mxfp4_linear(to[0], wt, y=y) is y and same(y, amd.mxfp4_linear(to[0], wt, out_dtype=F32))


def bound(x, w, want, terms, dtype):
    """How far an output may be off: see the top of the file."""
    S = x.abs() @ w.abs().t()
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    return (terms * 2.0 ** -23 * S) * (1 + torch.finfo(dtype).eps) + want.abs() * torch.finfo(dtype).eps / 2 + tiny


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (16, 100, 1501), (100, 333, 2048), (700, 900, 1000), (2456, 1300, 1911)])
def test_gemm_wide_scales(M, N, K):
    """Scales over 20 powers of two: sums that do round."""
    x, xt = random_rows(M, M, K, 117, 138)
    w, wt = random_rows(N, N, K, 117, 138)
    want = x @ w.t()
    for dtype in (BF, F32):
        got = amd.mxfp4_gemm(xt, wt, out_dtype=dtype).double()
        # one addition for every 64 of K and at most 16 pieces that are joined
        assert ((got - want).abs() <= bound(x, w, want, K / 64 + 17, dtype)).all()


@pytest.mark.parametrize("M,N,K", [(1, 100, 700), (16, 100, 700), (50, 2000, 300), (300, 300, 300), (2456, 3478, 300)])
def test_gemm_extreme_scales(M, N, K):
    """Products at both ends of fp32's range, and a NaN that stays in its row and its channel."""
    for low, xlow in ((240, 20), (1, 250), (0, 127)):
        x, xt = random_rows(3, M, K, xlow, xlow + 2)
        w, wt = random_rows(4, N, K, low, low + 2)
        assert same(amd.mxfp4_gemm(xt, wt, out_dtype=F32), (x @ w.t()).to(F32)), (low, xlow)
    x, xt = random_rows(5, M, K, 126, 128)
    w, wt = random_rows(6, N, K, 126, 128)
    codes, scales = wt.blocks()
    scales[7, 3] = 255
    wt = amd.Mxfp4Tensor.from_blocks(codes, scales, K)
    codes, scales = xt.blocks()
    scales[M // 2, -1] = 255
    y = amd.mxfp4_gemm(amd.Mxfp4Tensor.from_blocks(codes, scales, K), wt, out_dtype=F32)
    want = (x @ w.t()).to(F32)
    want[M // 2, :] = want[:, 7] = float("nan")
    assert same(y, want)


def test_gemm_without_K_and_empty():
    for M, N in ((3, 5), (300, 400)):
        x, w = (amd.Mxfp4Tensor(torch.zeros(n, 0, dtype=torch.uint8, device=dev()),
                                torch.zeros(0, dtype=torch.uint8, device=dev()), 0) for n in (M, N))
        y = torch.full((M, N), 7.0, device=dev())
        assert not amd.mxfp4_gemm(x, w, y=y).any()
        y.fill_(7.0)
        assert not amd.mxfp4_linear(torch.zeros(M, 0, device=dev()), w, y=y).any()
    _, w = random_rows(1, 5, 64)
    assert amd.mxfp4_linear(torch.zeros(0, 64, device=dev()), w).shape == (0, 5)
    assert amd.mxfp4_gemv(torch.zeros(0, 64, device=dev()), w).shape == (0, 5)
    y = torch.full((3, 5), 7.0, device=dev())
    w = amd.Mxfp4Tensor(torch.zeros(5, 0, dtype=torch.uint8, device=dev()), torch.zeros(0, dtype=torch.uint8, device=dev()), 0)
    assert not amd.mxfp4_gemv(torch.zeros(3, 0, device=dev()), w, y=y).any()


@pytest.mark.parametrize("M", [1, 20, 300])
def test_gemm_weights_past_4_gib(M):
    """Codes whose offsets pass 32 bits: the last channels are the ones of a small product."""
    K, N = 65536, 140000
    data = torch.zeros((N, K // 2), dtype=torch.uint8, device=dev())
    scale = torch.full((amd.mxfp4_scale_size(N, K),), 127, dtype=torch.uint8, device=dev())
    w, wt = random_rows(2, 64, K, 127, 128)
    data[-64:] = wt.data
    assert data.numel() > 1 << 32 and N % 32 == 0
    x, xt = random_rows(3, M, K, 127, 128)
    y = amd.mxfp4_gemm(xt, amd.Mxfp4Tensor(data, scale, K), out_dtype=F32)
    assert same(y[:, -64:], exactly(x, w, 0.25, F32)) and not y[:, :-64].any()
    if M == 1:
        v = torch.randint(-8, 9, (1, K), device=dev()).to(BF)
        y = amd.mxfp4_gemv(v, amd.Mxfp4Tensor(data, scale, K), out_dtype=F32)
        assert same(y[:, -64:], exactly(v.double(), w, 0.5, F32)) and not y[:, :-64].any()


# --- activations as they are -------------------------------------------------

@pytest.mark.parametrize("xdtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 4096), (2, 33, 31), (3, 100, 127), (4, 17, 1501), (5, 40, 11008),
                                   (7, 64, 4097), (8, 48, 129), (9, 20, 640), (16, 300, 2000), (16, 9000, 256), (1, 16, 70001),
                                   (3, 33000, 500), (5, 33000, 1000), (2, 33000, 2000), (16, 300, 9000),
                                   (4, 60, 15001), (7, 4500, 8300), (16, 9000, 4100), (3, 4200, 20003)])
def test_gemv(M, N, K, xdtype):
    """Exact for activations of few bits; within the bound for any."""
    g = torch.Generator(device=dev()).manual_seed(M + K)
    w, wt = random_rows(N, N, K, 127, 129)
    whole = torch.randint(-8, 9, (M * K + 1,), generator=g, device=dev())
    for shift in (0, 1):
        x = whole[shift:].to(xdtype)[:M * K].view(M, K) if shift == 0 else whole.to(xdtype)[1:].view(M, K)
        for dtype in TYPES:
            guard, y = guarded(M, N, dtype)
            amd.mxfp4_gemv(x, wt, y=y)
            assert same(y, exactly(x.double(), w, 0.5, dtype)) and untouched(guard, M * N)
    x = torch.randn(M, K, generator=g, device=dev()).to(xdtype)
    want = x.double() @ w.t()
    got = amd.mxfp4_gemv(x, wt, out_dtype=F32).double()
    # for every 32 of K an addition to each of three parts at most, eight waves' sums (or 16,
    # of a sixteenth of K each, with K of thousands)
    assert ((got - want).abs() <= bound(x.double(), w, want, 3 * K / 32 + 9, F32)).all()


@pytest.mark.parametrize("xdtype", TYPES, ids=str)
def test_gemv_takes_every_bit_of_an_activation(xdtype):
    """One activation and the weight 1: the output is the activation."""
    w = torch.zeros(8, 2, 16, dtype=torch.uint8, device=dev())
    w[:, 1, 3] = 2 << 4  # element 32 + 7
    t = amd.Mxfp4Tensor.from_blocks(w, torch.full((8, 2), 127, dtype=torch.uint8, device=dev()), 64)
    g = torch.Generator(device=dev()).manual_seed(3)
    for _ in range(20):
        x = torch.zeros(16, 64, device=dev(), dtype=xdtype)
        x[:, 39] = (torch.randn(16, generator=g, device=dev()) * torch.exp(torch.randn(16, generator=g, device=dev()) * 4)).to(xdtype)
        assert same(amd.mxfp4_gemv(x, t, out_dtype=F32), x[:, 39:40].float().expand(16, 8))


@pytest.mark.parametrize("xdtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(9, 40, 300), (7, 40, 9000), (16, 40, 9000)])
def test_gemv_not_finite(M, N, K, xdtype):
    """Infinities and NaN reach the outputs of their row alone."""
    w, wt = random_rows(1, N, K, 127, 128)
    x = torch.randint(-8, 9, (M, K), device=dev()).to(xdtype)
    x[2, 7], x[4, 299], x[5, 0], x[5, 1] = float("inf"), float("nan"), float("-inf"), torch.finfo(xdtype).max
    if xdtype == F32:  # a NaN whose upper half is an infinity's
        x.view(torch.int32)[6, 11] = 0x7F800001
    # products are fp32 numbers: the largest bf16 number times 1.5 or more passes 2^128 and is an
    # infinity, so with the -inf before it the sum is -inf or NaN by their signs, as that of the
    # products rounded to fp32 one by one
    want = (x.double()[:, None, :] * w[None]).to(F32).double().sum(2).to(F32)
    assert same(amd.mxfp4_gemv(x, wt, out_dtype=F32), want)
    y = amd.mxfp4_linear(x, wt, out_dtype=F32)
    bad = torch.tensor([2, 4, 5] + ([6] if xdtype == F32 else []), device=dev())
    assert y[bad].isnan().all() and y.isfinite().sum() == (M - len(bad)) * N


def test_gemv_refuses_many_rows():
    _, w = random_rows(1, 8, 64)
    with pytest.raises(ValueError, match="at most 16"):
        amd.mxfp4_gemv(torch.zeros(17, 64, device=dev()), w)


# --- rows sorted by expert ---------------------------------------------------

def routing(seed, T, k, E, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    if T > 3:
        ids[1], ids[2, 0] = E + 5, -7
    return ids


GROUPED = [(1, 2, 1, 8, 20), (5, 2, 3, 33, 300), (16, 4, 64, 40, 512), (1, 1, 1, 11, 4989), (1, 3, 1, 8, 11821),
           (18, 1, 1, 8, 16), (1687, 3, 1, 33, 17), (208, 3, 50, 163, 19), (1726, 3, 60, 285, 17), (134, 4, 1, 463, 6331),
           (596, 4, 1, 393, 2310), (586, 2, 3, 2466, 257), (1937, 3, 14, 981, 769), (586, 4, 10, 3044, 1568),
           (20, 2, 64, 900, 1100), (20, 2, 64, 1600, 600), (105, 3, 81, 645, 33), (20, 2, 64, 1600, 300)]


@pytest.mark.parametrize("T,k,E,N,K", GROUPED)
def test_grouped(T, k, E, N, K):
    x, xt = random_rows(T + K, T, K, 127, 129 if K < 10000 else 128)
    w, wt = random_rows(N + K, E * N, K, 127, 129 if K < 10000 else 128)
    ids = routing(T + N, T, k, E)
    route = amd.moe_sort(ids.to(dev()), E)
    offsets, order = route.offsets.cpu().tolist(), route.order.cpu().long()
    for dtype in TYPES:
        whole, y = guarded(T * k, N, dtype)
        amd.mxfp4_gemm_grouped(xt, wt, route, y=y)
        want = torch.full((T * k, N), 7.25, dtype=dtype, device=dev())
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                want[a:b] = exactly(x[(order[a:b] // k).to(dev())], w[e * N:(e + 1) * N], 0.25, dtype)
        assert same(y, want), f"{dtype}"
        assert untouched(whole, T * k * N)
    # one row to a sorted row
    n = offsets[E]
    sx, st = random_rows(5, T * k, K, 127, 128)
    y = amd.mxfp4_gemm_grouped(st, wt, route, out_dtype=F32, x_sorted=True)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            assert same(y[a:b], exactly(sx[a:b], w[e * N:(e + 1) * N], 0.25, F32))
    assert n <= T * k


@pytest.mark.parametrize("T,k,E,N,K", [(8, 2, 4, 50, 300), (208, 3, 5, 163, 190), (586, 4, 2, 3044, 260)])
def test_grouped_rows_without_a_source(T, k, E, N, K):
    """Orders past the tokens and negative ones give zeros, whatever the weights hold; bad offsets stay in range."""
    x, xt = random_rows(1, T, K, 127, 128)
    w, wt = random_rows(2, E * N, K, 127, 128)
    codes, scales = wt.blocks()
    scales[::7] = 255
    wt = amd.Mxfp4Tensor.from_blocks(codes, scales, K)
    w[::7] = float("nan")
    route = amd.moe_sort((torch.arange(T * k).view(T, k) % E).to(dev()), E)
    order = route.order.clone()
    order[3::5], order[4::11] = -1, T * k + 9
    bad = amd.MoeRoute(route.offsets, order, route.pos)
    y = amd.mxfp4_gemm_grouped(xt, wt, bad, out_dtype=F32)
    offsets = route.offsets.cpu().tolist()
    token = (order.long() // k).clamp(0, T - 1)
    gone = (order < 0) | (order >= T * k)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        want = (x[token[a:b]] @ w[e * N:(e + 1) * N].t()).to(F32)
        want[gone[a:b]] = 0.0
        assert same(y[a:b], want)
    wild = route.offsets.clone()
    wild[-1] = 1 << 30
    wild[1] = -5
    y = torch.full((T * k, N), 7.25, device=dev())
    amd.mxfp4_gemm_grouped(xt, wt, amd.MoeRoute(wild, route.order, route.pos), y=y)


# --- streams, graphs, order ---------------------------------------------------

SHAPES = [(1, 512, 4096), (13, 300, 1501), (69, 1856, 41721), (300, 300, 300), (700, 900, 1000), (2456, 3478, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_repeats_are_the_same_bits(M, N, K):
    g = torch.Generator(device=dev()).manual_seed(1)
    x = torch.randn(M, K, generator=g, device=dev())
    _, wt = random_rows(2, N, K, 110, 140)
    first = amd.mxfp4_linear(x, wt, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(amd.mxfp4_linear(x, wt, out_dtype=F32), first)
        if M <= 16:
            assert torch.equal(amd.mxfp4_gemv(x, wt, out_dtype=F32), amd.mxfp4_gemv(x, wt, out_dtype=F32))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_graphs_and_streams(M, N, K):
    """Two captured calls with workspaces of their own, replayed in turn with inputs that change, beside eager calls."""
    g = torch.Generator(device=dev()).manual_seed(4)
    _, wt = random_rows(2, N, K, 126, 129)
    xs = [torch.randn(M, K, generator=g, device=dev(), dtype=F32).to(BF) for _ in range(2)]
    ys = [torch.empty(M, N, device=dev()) for _ in range(2)]
    work = [amd.mxfp4_linear_workspace(M, N, K) for _ in range(2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for i in range(2):
            amd.mxfp4_linear(xs[i], wt, y=ys[i], workspace=work[i])
    torch.cuda.current_stream().wait_stream(stream)
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            amd.mxfp4_linear(xs[i], wt, y=ys[i], workspace=work[i])
        graphs.append(graph)
    for turn in range(4):
        for x in xs:
            x.copy_(torch.randn(M, K, generator=g, device=dev()))
        for y in ys:
            y.fill_(-1.0)
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        for x, y in zip(xs, ys):
            assert torch.equal(y, amd.mxfp4_linear(x, wt, out_dtype=F32))


def test_calls_on_two_streams_at_once():
    M, N, K = 300, 4096, 2048
    _, wt = random_rows(2, N, K, 126, 129)
    g = torch.Generator(device=dev()).manual_seed(4)
    xs = [torch.randn(M, K, generator=g, device=dev()) for _ in range(2)]
    want = [amd.mxfp4_linear(x, wt, out_dtype=F32) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[i].append(amd.mxfp4_linear(xs[i], wt, out_dtype=F32))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in out[i])
