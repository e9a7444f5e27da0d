"""GPU parity of the int8 encoder and products (include/int8.h) against the
definitions in 64 bits.

The codes and the integer sums are exact, and what follows them is a fixed
sequence of fp32 operations, so the results are compared bit for bit: scale =
fp32(a * fp32(1 / 127)), inverse = fp32(127 * fp32(1 / a)), code = rint of the
exact product x * inverse, output = fp32(fp32(fp32(sum) * xs) * ws) rounded once
to the output type."""
import numpy as np
import pytest
import torch

import w4a16_gemv_amd as amd

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF, FP, F32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def dev():
    return torch.device("cuda:0")


def same(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Equal bit for bit, any NaN equal to any other."""
    a, b = a.cpu(), b.cpu()
    nan = torch.isnan(a.float())
    if a.dtype != b.dtype or a.shape != b.shape or not torch.equal(nan, torch.isnan(b.float())):
        return False
    bits = {2: torch.int16, 4: torch.int32}[a.element_size()]
    z = torch.zeros((), dtype=a.dtype)
    return torch.equal(torch.where(nan, z, a).contiguous().view(bits),
                       torch.where(nan, z, b).contiguous().view(bits))


def encode(x: torch.Tensor):
    """(codes int64, scales fp32) of the rows of a CPU tensor, by definition."""
    v = x.double().numpy()
    finite = np.isfinite(v).all(1)
    a = np.abs(np.where(finite[:, None], v, 0.0)).max(1, initial=0.0)
    a = np.maximum(a, 2.0 ** -100).astype(np.float32)
    one = np.float32(1)
    inverse = (np.float32(127) * (one / a)).astype(np.float64)
    # both factors have 24 bits, so the fp64 product is exact; rint takes ties to even
    q = np.rint(np.where(finite[:, None], v, 0.0) * inverse[:, None]).astype(np.int64)
    return q, np.where(finite, a * (one / np.float32(127)), np.float32(np.nan)).astype(np.float32)


def padded(q: np.ndarray) -> torch.Tensor:
    rows, K = q.shape
    out = torch.zeros(rows, amd.int8_pitch(K), dtype=torch.int8)
    out[:, :K] = torch.from_numpy(q.astype(np.int8))
    return out


def random_tensor(rng, rows, K):
    """Codes over the whole range, -128 included, and scales; (q, scale, Int8Tensor)."""
    q = rng.integers(-128, 128, (rows, K))
    s = rng.uniform(0.5, 1.5, rows).astype(np.float32) * np.float32(2.0 ** -6)
    return q, s, amd.Int8Tensor(padded(q).to(dev()), torch.from_numpy(s).to(dev()), K)


def product(q, xs, w, ws, dtype):
    """The outputs by definition (numpy's fp32 products round one at a time)."""
    acc = (q.astype(np.float64) @ w.astype(np.float64).T).astype(np.float32)
    y = acc * xs.astype(np.float32)[:, None] * ws.astype(np.float32)[None, :]
    return torch.from_numpy(y).to(dtype)


GUARD = 96


def guarded(rows, N, dtype):
    """(whole buffer, view [rows][N] inside it); the rest holds a pattern."""
    whole = torch.full((rows * N + 2 * GUARD,), 7.25, dtype=dtype, device=dev())
    return whole, whole[GUARD:GUARD + rows * N].view(rows, N)


def untouched(whole, n):
    return bool((whole[:GUARD] == 7.25).all()) and bool((whole[GUARD + n:] == 7.25).all())


# --- the encoder -------------------------------------------------------------

QUANT = [(1, 1), (1, 7), (3, 8), (2, 63), (5, 64), (4, 65), (1, 4096), (7, 511), (9, 512), (3, 513), (2, 2047),
         (6, 2049), (3, 4099), (2, 8193), (2, 11008), (300, 33), (2, 16385), (1, 40001), (1, 131071), (1030, 128),
         (3, 12289), (2, 16384), (3, 20000), (2, 32768), (2, 32769), (1024, 2048), (2049, 1024), (2050, 70)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,K", QUANT)
def test_quantize(rows, K, dtype):
    g = torch.Generator().manual_seed(rows * 1000 + K)
    x = (torch.randn(rows, K, generator=g) * torch.rand(rows, 1, generator=g) * 5).to(dtype)
    x[0, K // 2] = 0.0
    # a row base that is aligned to nothing but the element
    room = torch.zeros(rows * K + 1, dtype=dtype, device=dev())
    for shift in (0, 1):
        view = room[shift:shift + rows * K].view(rows, K)
        view.copy_(x)
        t = amd.int8_quantize(view)
        q, s = encode(x)
        got = t.data.cpu()
        assert torch.equal(got, padded(q)), "codes or padding differ"
        assert same(t.scale, torch.from_numpy(s))
        for out in TYPES:
            v = torch.from_numpy(q.astype(np.float32) * s[:, None]).to(out)
            assert same(t.dequant(out_dtype=out), v)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_rounding_borders(dtype):
    """Rows whose values lie on and next to halves of a step: with peaks whose
    inverse is a power of two the ties are exact; with others the products come near."""
    rows = []
    for peak in (127.0, 254.0, 63.5, 1.0, 3.0, 96.0):
        step = peak / 127
        v = np.concatenate([[peak], step * (np.arange(-126, 126) + 0.5)])
        v = torch.tensor(v, dtype=torch.float64).to(dtype)
        for move in (0, 1, -1):
            w = v.clone()
            bits = w.view(torch.int32 if dtype == F32 else torch.int16)
            bits[1:] += move
            rows.append(w)
    x = torch.stack(rows)
    t = amd.int8_quantize(x.to(dev()))
    q, s = encode(x)
    assert torch.equal(t.data.cpu(), padded(q))
    assert same(t.scale, torch.from_numpy(s))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_extreme_rows(dtype):
    K = 130
    x = torch.zeros(9, K, dtype=dtype)
    top = torch.finfo(dtype).max
    x[1, 5], x[1, 6] = top, -top                          # the largest numbers
    x[2, :] = torch.finfo(dtype).smallest_normal
    x[3, 7] = torch.finfo(dtype).smallest_normal / 4      # subnormal
    x[4, 129] = float("inf")
    x[4, 0] = 1.0
    x[5, 64] = float("nan")
    x[6, 0], x[6, 1] = float("-inf"), float("nan")
    x[7, :] = -0.0
    x[8, :] = torch.linspace(-1, 1, K).to(dtype)
    t = amd.int8_quantize(x.to(dev()))
    q, s = encode(x)
    assert torch.equal(t.data.cpu(), padded(q))
    assert same(t.scale, torch.from_numpy(s))
    assert torch.isnan(t.scale.cpu()).tolist() == [False] * 4 + [True] * 3 + [False] * 2
    # only the outputs of those three rows are NaN
    _, _, w = random_tensor(np.random.default_rng(1), 20, K)
    y = amd.int8_gemm(t, w, out_dtype=F32).cpu()
    assert torch.isnan(y).all(1).tolist() == [False] * 4 + [True] * 3 + [False] * 2
    assert not torch.isnan(y[[0, 1, 2, 3, 7, 8]]).any()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_equals_the_tensor_expressions(dtype):
    """The codes and scales that a program gets from the same formulas in tensor
    operations on the device; every value here is near a half of the row's peak,
    where the quotient is next to a tie."""
    g = torch.Generator(device=dev()).manual_seed(5)
    x = torch.randn(4096, 96, generator=g, device=dev()).to(dtype)
    x[:, ::3] = x.abs().amax(1, keepdim=True) / 2
    a = x.float().abs().amax(1)
    q = (x.double() * (127.0 / a).double()[:, None]).round()
    t = amd.int8_quantize(x)
    assert torch.equal(t.data[:, :96].double(), q)
    assert same(t.scale, a / 127.0)


def test_quantize_shapes_and_out():
    x = torch.randn(2, 3, 70, device=dev())
    t = amd.int8_quantize(x)
    assert t.rows == 6 and t.K == 70 and t.nbytes == 6 * 128 + 24
    again = amd.int8_quantize(x * 2, out=t)
    assert again is t
    assert torch.equal(t.data.cpu(), padded(encode(x.cpu().view(6, 70))[0]))
    one = amd.int8_quantize(x[0, 0])
    assert one.rows == 1 and torch.equal(one.data[0], t.data[0])
    for empty in (torch.zeros(0, 70, device=dev()), torch.zeros(0, 0, device=dev())):
        assert amd.int8_quantize(empty).data.numel() == 0
    none = amd.int8_quantize(torch.zeros(3, 0, device=dev()))          # K = 0: scales alone
    assert none.data.shape == (3, 0)
    assert same(none.scale, torch.full((3,), 2.0 ** -100 / 127))
    with pytest.raises(ValueError, match="contiguous"):
        amd.int8_quantize(torch.zeros(8, 6, device=dev()).t())
    with pytest.raises(ValueError, match="expected 2 x 70"):
        amd.int8_quantize(x[0, :2], out=t)


# --- the product -------------------------------------------------------------

SIZES = [(1, 1, 1), (1, 17, 64), (1, 256, 4096), (2, 33, 65), (3, 100, 127), (5, 64, 1000), (8, 129, 2048),
         (9, 31, 63), (15, 16, 130), (16, 4099, 256), (17, 66, 513), (20, 130, 2), (31, 257, 128), (32, 64, 1024),
         (33, 65, 64), (48, 300, 200), (63, 7, 1501), (64, 512, 512), (65, 3, 300), (100, 1000, 64), (127, 129, 191),
         (128, 128, 128), (129, 255, 257), (200, 640, 4096), (255, 257, 500), (256, 256, 256), (257, 260, 320),
         (300, 1, 70), (513, 511, 129), (1, 11008, 300), (13, 1000, 4096), (700, 1030, 640)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm(M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    q, xs, x = random_tensor(rng, M, K)
    w, ws, wt = random_tensor(rng, N, K)
    for dtype in TYPES:
        whole, y = guarded(M, N, dtype)
        assert amd.int8_gemm(x, wt, y=y) is y
        assert same(y, product(q, xs, w, ws, dtype)), dtype
        assert untouched(whole, M * N)


@pytest.mark.parametrize("M,N,K", [(1, 130, 70000), (40, 40, 131071), (130, 70, 131071), (1, 20, 131071),
                                   (260, 260, 20000), (16, 100, 33333)])
def test_gemm_long_sums(M, N, K):
    """Sums near 2^31: every code -128 but for a few, so that nothing may overflow or be rounded."""
    q = np.full((M, K), -128)
    w = np.full((N, K), -128)
    q[:, ::97] = 127
    w[::2, ::101] = 5
    ones = lambda n: np.ones(n, np.float32)  # noqa: E731
    tensor = lambda a: amd.Int8Tensor(padded(a).to(dev()), torch.ones(len(a), device=dev()), K)  # noqa: E731
    y = amd.int8_gemm(tensor(q), tensor(w), out_dtype=F32)
    assert same(y, product(q, ones(M), w, ones(N), F32))


@pytest.mark.parametrize("M", [1, 4, 17, 64, 130, 260])
def test_gemm_workspace_does_not_change_the_bits(M):
    """A product that may split its sums over workgroups, with and without room to, and with a
    workspace that held other values."""
    N, K = 192, 8192
    rng = np.random.default_rng(M)
    q, xs, x = random_tensor(rng, M, K)
    w, ws, wt = random_tensor(rng, N, K)
    want = product(q, xs, w, ws, BF)
    work = amd.int8_gemm_workspace(M, N, K)
    room = [None, torch.zeros(256, dtype=torch.uint8, device=dev())]
    if work is not None:
        work.fill_(255)
        room += [work, work, torch.full((2 * work.numel() + 256,), 3, dtype=torch.uint8, device=dev())]
    for r in room:
        assert same(amd.int8_gemm(x, wt, workspace=r), want)


def test_gemm_padding_of_one_operand_may_hold_anything():
    rng = np.random.default_rng(5)
    M, N, K = 20, 150, 100
    q, xs, x = random_tensor(rng, M, K)
    w, ws, wt = random_tensor(rng, N, K)
    wt.data[:, K:] = 77
    assert same(amd.int8_gemm(x, wt), product(q, xs, w, ws, BF))


@pytest.mark.parametrize("M", [0, 1, 40])
@pytest.mark.parametrize("N", [0, 1, 70])
@pytest.mark.parametrize("K", [0, 64])
def test_gemm_empty_sizes(M, N, K):
    rng = np.random.default_rng(3)
    q, xs, x = random_tensor(rng, M, K)
    w, ws, wt = random_tensor(rng, N, K)
    y = amd.int8_gemm(x, wt, out_dtype=F32)
    assert y.shape == (M, N)
    if M * N:
        assert same(y + 0.0, product(q, xs, w, ws, F32) + 0.0)
    x16 = torch.randn(M, K, device=dev())
    z = amd.int8_linear(x16, wt, out_dtype=F32)
    assert same(z, amd.int8_gemm(amd.int8_quantize(x16), wt, out_dtype=F32))


def gpu_product(x, w, dtype):
    """product() on the GPU, for larger sizes: the fp64 sums of whole numbers are exact."""
    acc = x.data[:, :x.K].double() @ w.data[:, :w.K].double().t().contiguous()
    return (acc.float() * x.scale[:, None] * w.scale[None, :]).to(dtype)


# sizes for which each tiling is the fastest by the library's model, from the smallest tiles to the largest: whole
# turns, halves in a last turn, halves alone; and sums split over workgroups
TILINGS = [(17, 7, 64), (40, 500, 700), (33, 4099, 64), (120, 4100, 256), (100, 4099, 64), (128, 4096, 300), (200, 4099, 64),
           (513, 4100, 1000), (2049, 1000, 64), (1030, 4100, 640), (4100, 4099, 1501), (4096, 4096, 2048), (2000, 4001, 2048),
           (17, 7, 8192), (60, 64, 11000), (500, 30, 8192), (33, 1000, 8192), (65, 1000, 8192), (130, 513, 20000),
           (65, 2100, 8192), (18, 64, 131071), (33, 1500, 8192), (47, 1030, 4096), (48, 130, 4100),
           (17, 7, 12000), (17, 4099, 64), (250, 600, 11300), (1030, 7, 20000), (511, 260, 4100), (8191, 1, 64),
           (65, 1000, 40000), (65, 4099, 12000), (17, 2100, 8192),
           (4111, 4225, 1501), (4352, 4096, 1300), (8500, 2100, 1472)]


@pytest.mark.parametrize("M,N,K", TILINGS)
def test_gemm_tilings(M, N, K):
    rng = np.random.default_rng(M + N + K)
    _, _, x = random_tensor(rng, M, K)
    _, _, w = random_tensor(rng, N, K)
    for i, dtype in enumerate(TYPES):
        want = gpu_product(x, w, dtype)
        # the output aligned to nothing but its element in turn
        whole = torch.full((M * N + 2 * GUARD + 1,), 7.25, dtype=dtype, device=dev())
        y = whole[GUARD + i % 2:GUARD + i % 2 + M * N].view(M, N)
        amd.int8_gemm(x, w, y=y)
        assert same(y, want), dtype
        assert bool((whole[:GUARD + i % 2] == 7.25).all() and (whole[GUARD + i % 2 + M * N:] == 7.25).all())
        assert same(amd.int8_gemm(x, w, out_dtype=dtype, workspace=torch.empty(256, dtype=torch.uint8, device=dev())), want)


@pytest.mark.parametrize("M,N,K", [(1, 333, 700), (2, 64, 5000), (2, 50, 11264), (7, 333, 700), (16, 100, 2048), (16, 70, 4096), (5, 130, 11264),
                                   (13, 64, 11265), (90, 131, 700), (30, 64, 9000), (60, 64, 11300), (130, 1031, 700), (300, 1500, 130)])
def test_gemm_alignment(M, N, K):
    """Codes aligned to 16 bytes and no more, outputs to one element."""
    rng = np.random.default_rng(M * N + K)
    q, xs, x = random_tensor(rng, M, K)
    w, ws, wt = random_tensor(rng, N, K)

    def moved(t):
        room = torch.zeros(t.data.numel() + 16, dtype=torch.int8, device=dev())
        v = room[16:].view(t.data.shape)
        v.copy_(t.data)
        return amd.Int8Tensor(v, t.scale, t.K)

    for dtype in TYPES:
        whole = torch.full((M * N + 2 * GUARD + 1,), 7.25, dtype=dtype, device=dev())
        y = whole[GUARD + 1:GUARD + 1 + M * N].view(M, N)
        amd.int8_gemm(moved(x), moved(wt), y=y)
        assert same(y, product(q, xs, w, ws, dtype))
        assert bool((whole[:GUARD + 1] == 7.25).all() and (whole[GUARD + 1 + M * N:] == 7.25).all())


def test_offsets_past_32_bits():
    """Values, codes and outputs beyond the first 4 GiB (and 2^31 elements) of their tensors."""
    rows, K = 70000, 62000
    g = torch.Generator(device=dev()).manual_seed(3)
    x = torch.empty(rows, K, dtype=BF, device=dev())
    part = torch.randn(700, K, generator=g, device=dev()).to(BF)
    for i in range(0, rows, 700):
        x[i:i + 700] = part.roll(i // 700, 0)
    t = amd.int8_quantize(x)
    ends = [0, 1, 34639, 34640, 69998, 69999]
    q, s = encode(x[ends].cpu())
    assert torch.equal(t.data[ends].cpu(), padded(q)) and same(t.scale[ends], torch.from_numpy(s))
    assert same(t.dequant()[ends], torch.from_numpy(q.astype(np.float32) * s[:, None]).to(BF))
    del x
    few = amd.Int8Tensor(t.data[ends].contiguous(), t.scale[ends].contiguous(), K)
    y = amd.int8_gemm(few, t, out_dtype=F32)                    # 4.3 GB of weights
    assert same(y[:, ends], product(q, s, q, s, F32))
    y = amd.int8_gemm(t, few, out_dtype=F32)                    # of activations
    assert same(y[ends], product(q, s, q, s, F32))
    del t, y
    rng = np.random.default_rng(8)
    _, _, a = random_tensor(rng, 70000, 64)
    y = amd.int8_gemm(a, a)                                     # 9.8 GB of outputs
    b = amd.Int8Tensor(a.data[ends].contiguous(), a.scale[ends].contiguous(), 64)
    assert same(y[ends][:, ends], gpu_product(b, b, BF))
    assert same(y[:, ends], gpu_product(a, b, BF))


# --- quantize and product in one call ----------------------------------------

@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 4096), (1, 100, 11008), (2, 65, 300), (3, 17, 4097), (4, 300, 1501),
                                   (6, 64, 64), (8, 1000, 2048), (13, 77, 999), (16, 256, 8192), (33, 130, 513),
                                   (1, 50, 40000), (2, 40, 131071), (100, 70, 640), (333, 409, 1501)])
def test_linear_has_the_bits_of_the_two_calls(M, N, K):
    rng = np.random.default_rng(M + N + K)
    w, ws, wt = random_tensor(rng, N, K)
    for i, xdt in enumerate(TYPES):
        x = torch.from_numpy(rng.standard_normal((M, K))).to(xdt)
        x[M // 2, K // 3] *= 12
        q, xs = encode(x)
        room = torch.zeros(M * K + 1, dtype=xdt, device=dev())
        for shift, ydt in ((0, TYPES[i]), (1, TYPES[(i + 1) % 3])):
            view = room[shift:shift + M * K].view(M, K)
            view.copy_(x)
            whole, y = guarded(M, N, ydt)
            amd.int8_linear(view, wt, y=y)
            assert same(y, product(q, xs, w, ws, ydt))
            assert untouched(whole, M * N)


def test_linear_rows_that_are_not_finite():
    rng = np.random.default_rng(2)
    _, _, wt = random_tensor(rng, 90, 200)
    for M in (3, 40):
        x = torch.randn(M, 200, device=dev())
        x[1, 50], x[2, 0] = float("nan"), float("inf")
        y = amd.int8_linear(x, wt, out_dtype=F32).cpu()
        assert torch.isnan(y).all(1).tolist() == [i in (1, 2) for i in range(M)]
        assert not torch.isnan(y[[i for i in range(M) if i not in (1, 2)]]).any()


def test_linear_vector_and_method():
    rng = np.random.default_rng(4)
    w, ws, wt = random_tensor(rng, 70, 320)
    x = torch.randn(320, device=dev()).to(BF)
    y = amd.int8_linear(x, wt)
    assert y.shape == (70,)
    assert same(y, product(*encode(x.cpu()[None]), w, ws, BF)[0])
    out = torch.empty(70, device=dev())
    assert amd.int8_linear(x, wt, y=out) is out
    assert same(out, product(*encode(x.cpu()[None]), w, ws, F32)[0])
    assert same(wt.gemm(x[None]), y[None]) and same(wt.gemm(amd.int8_quantize(x[None])), y[None])
    work = amd.int8_linear_workspace(50, 70, 320)
    xx = torch.randn(50, 320, device=dev())
    assert same(amd.int8_linear(xx, wt, workspace=work), amd.int8_gemm(amd.int8_quantize(xx), wt))


def test_product_refusals():
    rng = np.random.default_rng(6)
    _, _, x = random_tensor(rng, 4, 100)
    _, _, w = random_tensor(rng, 6, 100)
    _, _, other = random_tensor(rng, 6, 90)
    with pytest.raises(ValueError, match="K=100"):
        amd.int8_gemm(x, other)
    with pytest.raises(ValueError, match="shape"):
        amd.int8_gemm(x, w, y=torch.empty(4, 7, device=dev()))
    with pytest.raises(ValueError, match="contiguous"):
        amd.int8_gemm(x, w, y=torch.empty(6, 4, device=dev()).t())
    with pytest.raises(ValueError, match="float32"):
        amd.int8_gemm(x, w, out_dtype=torch.float64)
    with pytest.raises(ValueError, match=r"\[M, 100\]"):
        amd.int8_linear(torch.zeros(4, 90, device=dev()), w)
    with pytest.raises(ValueError, match="expected cuda:0"):
        amd.int8_gemm(x, w, y=torch.empty(4, 6))
    _, _, long = random_tensor(rng, 2, 131072)
    with pytest.raises(amd.NF4Error) as e:
        amd.int8_gemm(long, long)
    assert e.value.status == amd.NF4_EUNSUPPORTED


# --- rows sorted by expert ---------------------------------------------------

def route_of(ids, E):
    """(offsets, order, pos) by definition."""
    flat = ids.reshape(-1)
    kept = [(int(e), i) for i, e in enumerate(flat) if 0 <= e < E]
    kept.sort()
    order = np.full(flat.size, -1, np.int32)
    pos = np.full(flat.size, -1, np.int32)
    for r, (_, i) in enumerate(kept):
        order[r], pos[i] = i, r
    offsets = np.searchsorted(np.array([e for e, _ in kept]), np.arange(E + 1)).astype(np.int32)
    return offsets, order, pos.reshape(ids.shape)


def to_route(arrays):
    return amd.MoeRoute(*(torch.from_numpy(np.ascontiguousarray(a)).to(dev()) for a in arrays))


def grouped(q, xs, w, ws, offsets, src, y0, dtype):
    """y0 with the experts' rows by definition; src: the row of q of each sorted row."""
    y = y0.clone()
    N = y0.shape[1]
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            y[a:b] = product(q[src[a:b]], xs[src[a:b]], w[e * N:(e + 1) * N], ws[e * N:(e + 1) * N], dtype)
    return y


@pytest.mark.parametrize("T,k,E,N,K,kind", [
    (1, 1, 1, 1, 1, "even"), (1, 2, 8, 100, 64, "even"), (3, 2, 5, 33, 65, "even"), (16, 4, 64, 128, 256, "even"),
    (40, 3, 7, 200, 300, "drop"), (64, 2, 100, 64, 130, "drop"), (100, 1, 1, 70, 513, "even"),
    (129, 2, 4, 300, 128, "one"), (300, 2, 8, 130, 1000, "skew"), (257, 4, 130, 40, 64, "drop"),
    (900, 2, 3, 260, 192, "skew"), (20, 2, 6, 17, 100, "none"), (64, 1, 1024, 16, 64, "even"),
    (700, 3, 9, 515, 320, "drop"), (2, 3, 4, 1000, 2048, "twice"), (5, 2, 4, 50, 0, "even")])
def test_gemm_grouped(T, k, E, N, K, kind):
    rng = np.random.default_rng(T + 10 * k + E + N + K)
    ids = rng.integers(0, E, (T, k))
    if kind == "drop":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[0] = E + 5
    elif kind == "one":
        ids[:] = 2
    elif kind == "skew":
        ids[rng.random((T, k)) < 0.7] = E - 1
    elif kind == "none":
        ids[:] = -1
    elif kind == "twice":
        ids[:] = ids[:, :1]
    q, xs, x = random_tensor(rng, T, K)
    w, ws, wt = random_tensor(rng, E * N, K)
    offsets, order, pos = route_of(ids, E)
    plan = to_route((offsets, order, pos))
    for dtype in TYPES:
        whole, y = guarded(T * k, N, dtype)
        want = grouped(q, xs, w, ws, offsets, order // k, y.cpu(), dtype)
        assert amd.int8_gemm_grouped(x, wt, plan, y=y) is y
        assert same(y, want), dtype
        assert untouched(whole, T * k * N)
    # activations in sorted order already
    q2, xs2, x2 = random_tensor(rng, T * k, K)
    whole, y = guarded(T * k, N, BF)
    want = grouped(q2, xs2, w, ws, offsets, np.arange(T * k), y.cpu(), BF)
    amd.int8_gemm_grouped(x2, wt, plan, y=y, x_sorted=True)
    assert same(y, want) and untouched(whole, T * k * N)


@pytest.mark.parametrize("rows,E,N,K", [(100, 1, 40, 64), (1500, 30, 130, 64), (900, 12, 1000, 256), (600, 1, 1030, 64), (6000, 1, 130, 64),
                                        (2700, 30, 515, 64), (6000, 30, 1030, 1024), (4500, 3, 2100, 1024), (9000, 2, 2048, 1500), (520, 64, 300, 128), (300, 30, 1000, 64),
                                        (200, 20, 130, 64), (1000, 64, 200, 192),
                                        (4400, 3, 4000, 1501), (8000, 2, 2300, 1500), (9300, 5, 2000, 1400)])
def test_gemm_grouped_tilings(rows, E, N, K):
    """Sizes of each tiling; uneven experts, slots dropped, k = 2."""
    rng = np.random.default_rng(rows + E + N)
    T = rows // 2
    ids = np.minimum(rng.geometric(2.0 / (E + 1), (T, 2)) - 1, E - 1)
    ids[rng.random((T, 2)) < 0.05] = -1
    _, _, x = random_tensor(rng, T, K)
    _, _, w = random_tensor(rng, E * N, K)
    offsets, order, pos = route_of(ids, E)
    plan = to_route((offsets, order, pos))
    for dtype in TYPES:
        whole, y = guarded(2 * T, N, dtype)
        amd.int8_gemm_grouped(x, w, plan, y=y)
        for e in range(E):
            a, b = int(offsets[e]), int(offsets[e + 1])
            token = torch.from_numpy(order[a:b] // 2).long().to(dev())
            xe = amd.Int8Tensor(x.data[token], x.scale[token], K)
            we = amd.Int8Tensor(w.data[e * N:(e + 1) * N], w.scale[e * N:(e + 1) * N], K)
            assert same(y[a:b], gpu_product(xe, we, dtype)), (dtype, e)
        assert bool((y[int(offsets[E]):] == 7.25).all()) and untouched(whole, 2 * T * N)


@pytest.mark.parametrize("T", [6, 200])
def test_gemm_grouped_survives_a_wrong_route(T):
    """Offsets and slots outside their ranges, or not ascending: nothing is read or written out of
    range, rows whose token does not exist are zeros."""
    rng = np.random.default_rng(T)
    E, N, K, k = 3, 70, 128, 2
    q, xs, x = random_tensor(rng, T, K)
    w, ws, wt = random_tensor(rng, E * N, K)
    order = np.arange(T * k, dtype=np.int32)
    order[1], order[2], order[3] = -1, 2 ** 31 - 1, T * k
    pos = np.zeros((T, k), np.int32)
    whole, y = guarded(T * k, N, F32)
    amd.int8_gemm_grouped(x, wt, to_route((np.array([0, T, T, 2 * T], np.int32), order, pos)), y=y)
    src = np.minimum(order // k, T - 1)
    zero = np.isin(np.arange(T * k), (1, 2, 3))
    want = grouped(q, np.where(zero[:T * k][:T], xs, xs), w, ws, [0, T, T, 2 * T], src, y.cpu() * 0, F32)
    want[torch.from_numpy(zero)] = 0.0
    assert same(y + 0.0, want + 0.0) and untouched(whole, T * k * N)
    for bad in ([0, -5, 10 ** 6, 3], [5, 2, 1, 0], [2 ** 31 - 1] * 4, [-2 ** 31] * 4):
        whole, y = guarded(T * k, N, F32)
        amd.int8_gemm_grouped(x, wt, to_route((np.array(bad, np.int32), order, pos)), y=y)
        torch.cuda.synchronize()
        assert untouched(whole, T * k * N)


def test_gemm_grouped_refusals():
    rng = np.random.default_rng(9)
    _, _, x = random_tensor(rng, 4, 64)
    _, _, w = random_tensor(rng, 10, 64)
    plan = to_route(route_of(np.zeros((4, 2), int), 3))
    with pytest.raises(ValueError, match="multiple of 3"):
        amd.int8_gemm_grouped(x, w, plan)
    _, _, w = random_tensor(rng, 9, 64)
    with pytest.raises(ValueError, match="expected 8"):
        amd.int8_gemm_grouped(x, w, plan, x_sorted=True)
    with pytest.raises(ValueError, match="shape"):
        amd.int8_gemm_grouped(x, w, plan, y=torch.empty(4, 3, device=dev()))
    _, _, w = random_tensor(rng, 9, 100)
    with pytest.raises(ValueError, match="K=64"):
        amd.int8_gemm_grouped(x, w, plan)


# --- streams and graphs ------------------------------------------------------

def test_two_streams_at_once():
    rng = np.random.default_rng(12)
    w, ws, wt = random_tensor(rng, 500, 3000)
    xs = [torch.randn(m, 3000, device=dev()) for m in (1, 24, 150, 400)]
    want = [amd.int8_linear(x, wt, out_dtype=F32) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(amd.int8_linear(x, wt, out_dtype=F32))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert same(a, b)


def test_captured_and_replayed():
    rng = np.random.default_rng(13)
    w, ws, wt = random_tensor(rng, 300, 2000)
    for M in (1, 8, 40, 200):
        x = torch.randn(M, 2000, device=dev())
        amd.int8_linear(x, wt)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t = amd.int8_quantize(x)
            y = amd.int8_gemm(t, wt, out_dtype=F32)
            z = amd.int8_linear(x, wt, out_dtype=F32)
        for i in range(4):
            x.normal_()
            want = product(*encode(x.cpu()), w, ws, F32)
            y.zero_(), z.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same(y, want) and same(z, want)
            assert same(amd.int8_linear(x, wt, out_dtype=F32), want)


def test_captured_split_product():
    """A product whose sums are split over workgroups, two kernels, replayed with other codes."""
    rng = np.random.default_rng(19)
    M, N, K = 128, 1024, 11008
    assert amd.load().int8_gemm_workspace_size(M, N, K) > 0
    _, _, w = random_tensor(rng, N, K)
    x = amd.int8_quantize(torch.randn(M, K, device=dev()))
    amd.int8_gemm(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = amd.int8_gemm(x, w)
    for _ in range(4):
        amd.int8_quantize(torch.randn(M, K, device=dev()), out=x)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(y, gpu_product(x, w, BF))
        assert same(amd.int8_gemm(x, w), y)


def test_captured_grouped_tiles_follow_the_routing():
    """Large tiles of a captured product: how many there are, and whether the last turn's are computed
    whole, in halves or in quarters, follows each replay's routing."""
    T, k, E, N, K = 2200, 2, 3, 4000, 1501
    rng = np.random.default_rng(23)
    _, _, w = random_tensor(rng, E * N, K)
    _, _, x = random_tensor(rng, T, K)
    ids = torch.from_numpy(rng.integers(0, E, (T, k))).to(dev())

    def run(y):
        plan = amd.moe_sort(ids, E)
        return plan, amd.int8_gemm_grouped(x, w, plan, y=y)

    y = torch.empty(T * k, N, dtype=BF, device=dev())
    run(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, _ = run(y)
    # tokens routed, and the share of slots sent to the first expert: from 18 row tiles (of 16 channel tiles) to none
    for routed, share in ((T, 0.0), (T, 1.0), (1100, 0.0), (1650, 0.5), (3, 0.0), (0, 0.0)):
        ids.random_(0, E)
        ids[torch.rand(T, k, device=dev()) < share] = 0
        ids[routed:] = -1
        y.fill_(7.25)
        graph.replay()
        torch.cuda.synchronize()
        offsets = plan.offsets.tolist()
        assert offsets[E] == routed * k
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            token = plan.order[a:b].long() // k
            xe = amd.Int8Tensor(x.data[token], x.scale[token], K)
            we = amd.Int8Tensor(w.data[e * N:(e + 1) * N], w.scale[e * N:(e + 1) * N], K)
            assert same(y[a:b], gpu_product(xe, we, BF)), (routed, e)
        assert bool((y[offsets[E]:] == 7.25).all())
        again = torch.full_like(y, 7.25)
        run(again)
        assert same(again, y)
