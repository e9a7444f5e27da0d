"""What the headers and docstrings of the int8 products and of the routing promise
beyond the values themselves, on the GPU."""
import ctypes as C

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import w4a16_gemv_amd as amd
from tests import test_gpu_moe
from tests.test_gpu_int8 import (BF, F32, TYPES, dev, encode, gpu_product, guarded, padded, product, random_tensor, route_of, same,
                                 to_route, untouched)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def plan(M, N, K, experts=0, room=1 << 62):
    """(plan, detail) of include/nf4_probe.h: the kernel and variant that these sizes go to."""
    a, b = C.c_int32(), C.c_int32()
    assert amd.load().nf4_probe_int8_plan(M, N, K, experts, room, C.byref(a), C.byref(b)) == 0
    return a.value, b.value


DOT, ROWS, LARGEST = -2, -1, 5

# --- workspaces --------------------------------------------------------------

# products that split K over workgroups: every tiling that does
SPLITS = [(17, 7, 12000), (18, 64, 131071), (130, 513, 20000), (1030, 7, 20000), (250, 600, 11300), (17, 2100, 8192),
          (65, 1000, 8192), (65, 1000, 40000), (65, 4099, 12000), (128, 1024, 11008)]


@pytest.mark.parametrize("M,N,K", SPLITS)
def test_split_products_in_any_workspace(M, N, K):
    """The bits with room for all pieces of K, for more, for fewer and for none; workspaces that held other values
    and are not written past the pieces that fit."""
    rng = np.random.default_rng(M + N + K)
    _, _, x = random_tensor(rng, M, K)
    _, _, w = random_tensor(rng, N, K)
    plane = M * ((N + 3) // 4 * 4) * 4
    splits = plan(M, N, K)[1]
    work = amd.int8_gemm_workspace(M, N, K)
    assert splits > 1 and work is not None and work.numel() == splits * plane
    want = gpu_product(x, w, F32)
    used = set()
    for room in (work.numel(), work.numel() - 1, 2 * work.numel() + 256, (splits - 1) * plane, 2 * plane, plane, 256):
        whole = torch.full((room + 256,), 255, dtype=torch.uint8, device=dev())
        pieces = plan(M, N, K, room=room)[1]
        assert pieces == 1 or pieces * plane <= room
        used.add(pieces)
        for _ in range(2):
            assert same(amd.int8_gemm(x, w, out_dtype=F32, workspace=whole[:room]), want), room
        edge = pieces * plane if pieces > 1 else 0
        assert bool((whole[edge:] == 255).all()), room
    assert len(used) > 1
    assert same(amd.int8_gemm(x, w, out_dtype=F32), want)
    # and in a workspace of int8_linear, behind the codes
    a = torch.randn(M, K, device=dev())
    work = amd.int8_linear_workspace(M, N, K)
    work.fill_(255)
    assert same(amd.int8_linear(a, w, workspace=work), gpu_product(amd.int8_quantize(a), w, BF))


@pytest.mark.parametrize("larger,shapes", [
    ((139, 512, 8192), [(139, 512, 8192), (138, 512, 8192), (130, 512, 8000), (40, 512, 4097), (2, 512, 64), (1, 512, 0)]),
    ((311, 512, 11008), [(310, 512, 11008), (128, 1024, 11008), (17, 4099, 300)]),
    ((622, 256, 11008), [(621, 256, 11008), (65, 1000, 11000)])])
def test_linear_takes_the_workspace_of_a_larger_shape(larger, shapes):
    """A smaller M may split its sums more and so could use more room than the larger one has."""
    work = amd.int8_linear_workspace(*larger)
    assert any(amd.load().int8_linear_workspace_size(*s) > work.numel() for s in shapes)
    rng = np.random.default_rng(sum(larger))
    for M, N, K in shapes:
        w, ws, wt = random_tensor(rng, N, K)
        x = torch.from_numpy(rng.standard_normal((M, K))).to(BF)
        work.fill_(255)
        whole = torch.cat([work, torch.full((256,), 7, dtype=torch.uint8, device=dev())])
        y = amd.int8_linear(x.to(dev()), wt, out_dtype=F32, workspace=whole[:work.numel()])
        assert same(y + 0.0, product(*encode(x), w, ws, F32) + 0.0), (M, N, K)
        assert bool((whole[work.numel():] == 7).all())


# --- gradients ---------------------------------------------------------------

def test_learned_scales_under_no_grad():
    rng = np.random.default_rng(3)
    q, xs, x = random_tensor(rng, 5, 130)
    w, ws, wt = random_tensor(rng, 40, 130)
    wt.scale.requires_grad_()
    for call in (lambda: amd.int8_gemm(x, wt, out_dtype=F32), lambda: amd.int8_gemm(wt, x, out_dtype=F32),
                 lambda: amd.int8_linear(torch.ones(3, 130, device=dev()), wt), lambda: wt.dequant()):
        with pytest.raises(ValueError, match="scale requires a gradient"):
            call()
    with torch.no_grad():
        assert same(amd.int8_gemm(x, wt, out_dtype=F32), product(q, xs, w, ws, F32))

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, scale):
            ctx.save_for_backward(scale)
            return amd.int8_gemm(x, amd.Int8Tensor(wt.data, scale, 130), out_dtype=F32)

        @staticmethod
        def backward(ctx, g):
            scale, = ctx.saved_tensors
            return (g * amd.int8_gemm(x, amd.Int8Tensor(wt.data, torch.ones_like(scale), 130), out_dtype=F32)).sum(0)

    y = Product.apply(wt.scale)                # inside a Function nothing is being recorded
    y.backward(torch.ones_like(y))
    assert same(y.detach(), product(q, xs, w, ws, F32)) and wt.scale.grad is not None


def test_forward_mode():
    rng = np.random.default_rng(4)
    _, _, wt = random_tensor(rng, 40, 96)
    x, dx = torch.ones(3, 96, device=dev()), torch.randn(3, 96, device=dev())
    want = amd.int8_linear(x, wt, out_dtype=F32)
    route = amd.moe_sort(torch.tensor([[0], [1], [0]], device=dev()), 2)

    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return amd.moe_gather(x, route)

        @staticmethod
        def jvp(ctx, t):
            return amd.moe_gather(t, route)

    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, dx)
        for call in (lambda: amd.int8_linear(dual, wt), lambda: amd.int8_quantize(dual),
                     lambda: amd.moe_gather(dual, route), lambda: amd.moe_combine(dual, route)):
            with pytest.raises(ValueError, match="tangent"):
                call()
        assert same(amd.int8_linear(x, wt, out_dtype=F32), want)          # others go on as before
        out = forward_ad.unpack_dual(Gather.apply(dual))
        assert same(out.primal, x) and same(out.tangent, dx[[0, 2, 1]])


# --- roundings ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_encoder_against_quotients_in_64_bits(dtype):
    """Scales, codes and values against a / 127, 127 x / a and x, over the whole range of peaks.

    1 / a and the product with 127 are rounded once each, 2^-24 relative: 127 (2^-23 + 2^-48) < 2^-16 in a code.  For
    a > 2^126 1 / a is a multiple of 2^-149 above 2^-128, 2^-22 relative, in all 127 (2^-22 + 2^-24 + 2^-46) < 2^-14.  A
    value adds the scale's two roundings, 127 (2^-23 + 2^-48) more, and the product's, 127 2^-24."""
    g = torch.Generator().manual_seed(11)
    top = np.log2(torch.finfo(dtype).max)
    rows, K = 6000, 96
    exponent = torch.rand(rows, 1, generator=g, dtype=torch.float64) * (top + 99) - 99
    exponent[:2000] = top - torch.rand(2000, 1, generator=g, dtype=torch.float64) * 2     # 1 / a may be subnormal
    x = torch.rand(rows, K, generator=g, dtype=torch.float64) * 2 - 1
    x[:, 0] = 1.0
    x[:, 1::7] = torch.randint(-254, 255, (rows, 14), generator=g).double() / 254              # next to ties
    x = (x * torch.exp2(exponent - 2.0 ** -20)).to(dtype)
    t = amd.int8_quantize(x.to(dev()))
    v, q, scale = x.double().numpy(), t.data[:, :K].cpu().double().numpy(), t.scale.cpu().double().numpy()
    assert np.isfinite(v).all() and np.isfinite(scale).all()
    a = np.maximum(np.abs(v).max(1), 2.0 ** -100)
    high = (a > 2.0 ** 126)[:, None]
    assert (np.abs(scale - a / 127) <= a / 127 * (2.0 ** -23 + 2.0 ** -47)).all()
    slack = np.where(high, 2.0 ** -14, 2.0 ** -16)
    assert (np.abs(q - 127 * v / a[:, None]) <= 0.5 + slack).all()
    got = t.dequant(out_dtype=F32).cpu().double().numpy()
    assert (np.abs(got - v) <= (0.5 + np.where(high, 2.0 ** -13, 2.0 ** -14)) * a[:, None] / 127).all()
    assert dtype == torch.float16 or (high.any() and not high.all())


@pytest.mark.parametrize("M,N", [(1, 40), (2, 33), (7, 300), (40, 700), (300, 1030), (600, 2100)])
def test_three_fp32_roundings_in_order(M, N):
    """fp32(fp32(fp32(sum) xs) ws): within (1 + 2^-24)^3 of the exact value where both products are normal; past
    fp32's range and below its normal numbers the first product has the last word."""
    rng = np.random.default_rng(M)
    K = 320
    q, _, x = random_tensor(rng, M, K)
    w, _, wt = random_tensor(rng, N, K)
    xs = (2.0 ** rng.uniform(-148, 127, M)).astype(np.float32)
    ws = (2.0 ** rng.uniform(-148, 127, N)).astype(np.float32)
    xs[0], ws[:3] = 2.0 ** 126, (2.0 ** -100, 2.0 ** -140, 2.0 ** 3)
    x.scale.copy_(torch.from_numpy(xs)), wt.scale.copy_(torch.from_numpy(ws))
    got = amd.int8_gemm(x, wt, out_dtype=F32).cpu()
    with np.errstate(over="ignore"):
        assert same(got, product(q, xs, w, ws, F32))
        acc = q.astype(np.float64) @ w.astype(np.float64).T
        first = acc.astype(np.float32) * xs[:, None]
    exact = acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    got = got.double().numpy()
    tiny, top = 2.0 ** -126, float(np.finfo(np.float32).max)
    normal = lambda a: (np.abs(a) >= tiny) & (np.abs(a) <= top)  # noqa: E731
    good = (normal(first) & normal(got)) | (acc == 0)
    assert (np.abs(got - exact)[good] <= np.abs(exact)[good] * ((1 + 2.0 ** -24) ** 3 - 1 + 2.0 ** -50)).all()
    out = np.isinf(first)
    assert out[0].any() and (M == 1 or good.any()) and np.isinf(got[out]).all() and (np.abs(exact[out]) < top).any()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,K", [(1, 4096), (3, 4097), (300, 4160), (2, 6145), (5, 8191), (1200, 8192), (2, 8193), (3, 12288), (2, 12289), (2, 16385)])
def test_encoder_on_both_sides_of_each_variant(rows, K, dtype):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K, generator=g) * 3).to(dtype)
    x[:, -1] = x.abs().amax(1) * 2                      # the peak in the last piece
    room = torch.zeros(rows * K + 1, dtype=dtype, device=dev())
    for shift in (0, 1):
        view = room[shift:shift + rows * K].view(rows, K)
        view.copy_(x)
        t = amd.Int8Tensor(torch.full((rows, amd.int8_pitch(K)), 85, dtype=torch.int8, device=dev()), torch.zeros(rows, device=dev()), K)
        amd.int8_quantize(view, out=t)
        q, s = encode(x)
        assert torch.equal(t.data.cpu(), padded(q)) and same(t.scale, torch.from_numpy(s))


# --- every kernel ------------------------------------------------------------

# (plan, detail) and sizes: variants that the sizes of test_gpu_int8.py leave out, and one of each other kind
KERNELS = [((DOT, 4), (1, 100, 1000)), ((DOT, 8), (2, 77, 7000)), ((DOT, 8), (1, 130, 8001)), ((DOT, 11), (2, 50, 11201)),
           ((ROWS, 4), (5, 130, 1000)), ((ROWS, 8), (13, 100, 4000)), ((ROWS, 22), (16, 100, 11201)),
           ((0, 1), (128, 4096, 300)), ((1, 1), (33, 4099, 60)), ((2, 1), (100, 4099, 60)), ((3, 1), (200, 4099, 60)),
           ((4, 1), (2049, 1000, 60)), ((0, 11), (17, 7, 12000)), ((2, 8), (65, 1000, 8190)),
           ((LARGEST, 2), (2000, 4001, 2030)), ((LARGEST, 3), (4600, 5000, 1500)), ((LARGEST, 5), (4100, 4099, 1501))]


@pytest.mark.parametrize("kind,size", KERNELS)
def test_padding_of_either_operand_may_hold_anything(kind, size):
    M, N, K = size
    assert plan(M, N, K) == kind and K % 64
    rng = np.random.default_rng(M + N + K)
    for side in (0, 1):
        _, _, x = random_tensor(rng, M, K)
        _, _, w = random_tensor(rng, N, K)
        want = gpu_product(x, w, BF)
        t = (x, w)[side]
        t.data[:, K:] = torch.from_numpy(rng.integers(-128, 128, (t.rows, t.data.shape[1] - K)).astype(np.int8)).to(dev())
        assert same(amd.int8_gemm(x, w), want)
        assert same(amd.int8_gemm(x, w, workspace=torch.empty(256, dtype=torch.uint8, device=dev())), want)


# both sides of what sends few rows to the few-row kernel: the kernel and the size
FEW = [(ROWS, (16, 4096, 4150)), (0, (16, 4097, 4150)), (0, (3, 8192, 8192)), (ROWS, (3, 8193, 8130)), (0, (3, 8193, 8120)),
       (ROWS, (16, 12000, 11264)), (0, (16, 4500, 11265)), (ROWS, (16, 9000, 4096)), (ROWS, (17, 4096, 4096)), (0, (17, 2100, 4097))]


@pytest.mark.parametrize("kernel,size", FEW)
def test_both_sides_of_the_few_row_rule(kernel, size):
    M, N, K = size
    rng = np.random.default_rng(M + N + K)
    _, _, x = random_tensor(rng, M, K)
    _, _, w = random_tensor(rng, N, K)
    assert (plan(M, N, K)[0] == ROWS) == (kernel == ROWS)
    for dtype in TYPES:
        whole, y = guarded(M, N, dtype)
        amd.int8_gemm(x, w, y=y)
        assert same(y, gpu_product(x, w, dtype)) and untouched(whole, M * N)
    a = torch.randn(M, K, device=dev())
    assert same(amd.int8_linear(a, w), gpu_product(amd.int8_quantize(a), w, BF))


# (plan, detail) and (rows, experts, N, K)
GROUPED = [((ROWS, 4), (120, 40, 70, 1000)), ((ROWS, 8), (60, 20, 100, 4000)), ((ROWS, 22), (60, 20, 100, 11000)),
           ((ROWS, 22), (8, 8, 515, 8300)), ((0, 1), (100, 1, 40, 60)), ((1, 1), (1500, 30, 130, 60)), ((2, 1), (600, 1, 1030, 60)),
           ((3, 1), (900, 12, 1000, 250)), ((4, 1), (2700, 30, 515, 60)), ((LARGEST, 1), (4400, 3, 4000, 1501)),
           ((2, 1), (8, 8, 4096, 8100)), ((2, 1), (32, 16, 515, 9000)), ((0, 1), (8, 8, 515, 4200)),
           ((ROWS, 22), (60, 20, 2910, 8150)), ((2, 1), (60, 20, 2800, 8150)),
           ((LARGEST, 1), (8000, 2, 2300, 1500)), ((LARGEST, 1), (9300, 5, 2000, 1400))]


@pytest.mark.parametrize("x_sorted", [False, True])
@pytest.mark.parametrize("kind,size", GROUPED)
def test_gemm_grouped_kernels(kind, size, x_sorted):
    """Each kernel with the tokens' rows in either order, padding that holds anything, and uneven experts."""
    rows, E, N, K = size
    assert plan(rows, N, K, E) == kind and K % 64
    rng = np.random.default_rng(rows + E + N)
    T = rows // 2
    ids = np.minimum(rng.geometric(2.0 / (E + 1), (T, 2)) - 1, E - 1)
    ids[rng.random((T, 2)) < 0.05] = -1
    _, _, x = random_tensor(rng, rows if x_sorted else T, K)
    _, _, w = random_tensor(rng, E * N, K)
    offsets, order, pos = route_of(ids, E)
    route = to_route((offsets, order, pos))
    source = torch.arange(rows, device=dev()) if x_sorted else route.order.long().clamp_min(0) // 2
    want = torch.full((rows, N), 7.25, dtype=BF, device=dev())
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        xe = amd.Int8Tensor(x.data[source[a:b]], x.scale[source[a:b]], K)
        we = amd.Int8Tensor(w.data[e * N:(e + 1) * N], w.scale[e * N:(e + 1) * N], K)
        want[a:b] = gpu_product(xe, we, BF)
    for t in (None, x, w):
        if t is not None:
            kept = t.data[:, K:].clone()
            t.data[:, K:] = 93
        whole, y = guarded(rows, N, BF)
        amd.int8_gemm_grouped(x, w, route, y=y, x_sorted=x_sorted)
        assert same(y, want) and untouched(whole, rows * N)
        if t is not None:
            t.data[:, K:] = kept


# --- rows sorted by expert ---------------------------------------------------

# by kernel: few rows, tiles of several sizes, the largest with a last turn in halves and in quarters
ABSENT = [(6, 2, 3, 70, 128), (100, 2, 2, 40, 64), (200, 2, 3, 70, 128), (600, 2, 4, 515, 64), (1500, 2, 2, 1030, 300),
          (2200, 2, 3, 4000, 130), (4650, 2, 5, 2000, 140), (4000, 2, 2, 2300, 150),
          (2200, 2, 3, 4000, 1500), (4650, 2, 5, 2000, 1400), (4000, 2, 2, 2300, 1500), (8, 2, 5, 70, 4000), (8, 2, 5, 70, 9000)]


@pytest.mark.parametrize("T,k,E,N,K", ABSENT)
def test_rows_without_a_token_are_zeros_beside_scales_that_are_not_finite(T, k, E, N, K):
    """A slot of a token that does not exist, and channels that the encoder marked as not finite (NaN scale)."""
    rng = np.random.default_rng(T + N)
    _, _, x = random_tensor(rng, T, K)
    _, _, w = random_tensor(rng, E * N, K)
    bad = torch.from_numpy(rng.random(E * N) < 0.2).to(dev())
    bad[:2] = True
    w.scale[bad] = float("nan")
    w.scale[1], w.scale[2] = float("inf"), -w.scale[2]
    order = rng.permutation(T * k).astype(np.int32)
    gone = rng.random(T * k) < 0.1
    gone[:3] = True
    order[gone] = rng.choice(np.array([-1, -2 ** 31, T * k, 2 ** 31 - 1], np.int32), gone.sum())
    offsets = np.linspace(0, T * k, E + 1).astype(np.int32)
    plan = to_route((offsets, order, np.zeros((T, k), np.int32)))
    gone = torch.from_numpy(gone).to(dev())
    for dtype in TYPES:
        whole, y = guarded(T * k, N, dtype)
        amd.int8_gemm_grouped(x, w, plan, y=y)
        assert bool((y[gone].float() == 0).all()) and untouched(whole, T * k * N), dtype
        for e in range(E):
            rows = torch.arange(int(offsets[e]), int(offsets[e + 1]), device=dev())
            rows = rows[~gone[rows]]
            token = plan.order[rows].long() // k
            xe = amd.Int8Tensor(x.data[token], x.scale[token], K)
            we = amd.Int8Tensor(w.data[e * N:(e + 1) * N], w.scale[e * N:(e + 1) * N], K)
            assert same(y[rows], gpu_product(xe, we, dtype)), (dtype, e)


# --- routing -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,kind", [(1024, 1, 5, 513, "drop"), (1025, 1, 5, 513, "drop"), (1024, 2, 9, 1024, "all"), (1025, 2, 9, 1024, "all"),
                                          (1030, 5, 7, 1001, "drop"), (257, 2, 8, 1001, "all"), (1100, 1, 3, 512, "drop")])
def test_rows_of_few_and_many_tokens(T, k, E, H, kind, dtype):
    """On both sides of the number of tokens at which a token's row goes to a wave instead of a workgroup."""
    test_gpu_moe.test_gather(T, k, E, H, kind, dtype)
    test_gpu_moe.test_combine(T, k, E, H, kind, dtype)
    test_gpu_moe.test_combine_grad(T, k, E, H, kind, dtype)
