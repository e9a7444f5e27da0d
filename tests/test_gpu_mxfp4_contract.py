"""What include/mxfp4.h promises beside the values themselves: bytes that may hold
anything, experts that leave each other alone; and the variants of its kernels."""
import ctypes as C

import pytest
import torch

import w4a16_gemv_amd as amd
from tests.test_gpu_mxfp4 import F32, TYPES, dev, exactly, guarded, plan, random_rows, same, untouched
from tests.test_gpu_mxfp4_mlp import check, make

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def padded(t):
    """t with the scales of the rows past its last, which may hold anything, those of NaN."""
    scale = t.scale.clone()
    tiles = scale.view(-(-t.rows // 32), -1, 2, 32, 4)
    assert t.rows % 32
    tiles[-1, :, :, t.rows % 32:] = 255
    return amd.Mxfp4Tensor(t.data, scale, t.K)


def bits(a, b):
    """Equal bit for bit."""
    as_int = torch.int32 if a.dtype == F32 else torch.int16
    return torch.equal(a.view(as_int), b.view(as_int))


# --- rows whose step of sixteen units has no room in LDS ------------------------

# 14 to 16 rows in fp16 or 10 to 16 in fp32 of 257 to 512 elements, where four waves share a row
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(16, 40, 400), (14, 100, 512), (10, 33, 257), (12, 700, 384), (16, 3000, 500)])
def test_gemv_nan_stays_in_its_row(M, N, K, dtype):
    """Rows stand side by side in LDS; what a wave reads past one must not be the next."""
    w, wt = random_rows(N, N, K, 127, 129)
    x = torch.randint(-8, 9, (M, K), device=dev()).to(dtype)
    want = exactly(x.double(), w, 0.5, F32)
    assert same(amd.mxfp4_gemv(x, wt, out_dtype=F32), want)
    for row in (1, M // 2, M - 1):
        hurt, some = x.clone(), want.clone()
        hurt[row], some[row] = NAN, NAN
        assert same(amd.mxfp4_gemv(hurt, wt, out_dtype=F32), some)


@pytest.mark.parametrize("gated", (True, False), ids=("gated", "plain"))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", [(20, 3, 5, 257, 41), (16, 1, 1, 400, 60), (64, 2, 3, 512, 33), (13, 2, 2, 384, 64)])
def test_mlp_rows_of_257_to_512(T, k, E, H, F, dtype, gated):
    x, w1, t1, w2, t2, ids, weights = make(T + F, T, k, E, H, F, gated, dtype)
    check(amd.mxfp4_moe_mlp(x, t1, t2, ids, weights), x, w1, w2, ids, weights, E, gated)


# --- every way to take rows ------------------------------------------------------

def rows_plan(T, k, E, H, F, dtype):
    """include/nf4_probe.h's plan of rows (needs no GPU): waves, units, elements in LDS, rows, way down."""
    a = (C.c_int32 * 5)()
    assert amd.load().nf4_probe_mxfp4_rows(T, k, E, H, F, TYPES.index(dtype), a) == 0
    return tuple(a)


# rows, channels, K
GEMV = [(1, 40, 100), (1, 17000, 300), (1, 40, 300), (1, 40, 600), (14, 40, 300), (10, 40, 300), (1, 40, 1200), (1, 40, 2600),
        (3, 40, 20000), (4, 40, 4200), (3, 40, 4200), (7, 40, 4200), (7, 40, 2600), (5, 40, 2600), (14, 40, 2600),
        (14, 40, 1200), (10, 40, 1200)]
# tokens, slots, experts, H, F
MLP = [(1, 1, 1, 100, 40), (8, 8, 64, 300, 130), (64, 8, 64, 2600, 40), (1, 1, 1, 300, 40), (1, 1, 1, 600, 40),
       (16, 1, 1, 2600, 40), (1, 1, 1, 1200, 40), (8, 1, 1, 4200, 40), (1, 1, 1, 2600, 40), (3, 1, 1, 4200, 40),
       (64, 8, 64, 1200, 130), (40, 8, 64, 1200, 130), (16, 1, 1, 1200, 40), (16, 1, 1, 300, 40), (8, 1, 1, 2600, 40),
       (3, 1, 1, 9000, 40), (8, 8, 64, 2600, 40), (8, 8, 64, 2200, 40), (20, 4, 64, 100, 40), (8, 1, 1, 100, 40),
       (20, 1, 1, 100, 40), (1, 2, 8, 2048, 50)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", GEMV)
def test_gemv_variants(M, N, K, dtype):
    w, wt = random_rows(N, N, K, 127, 129)
    x = torch.randint(-8, 9, (M, K), device=dev()).to(dtype)
    for out in TYPES:
        whole, y = guarded(M, N, out)
        amd.mxfp4_gemv(x, wt, y=y)
        assert same(y, exactly(x.double(), w, 0.5, out)) and untouched(whole, M * N)


@pytest.mark.parametrize("gated", (True, False), ids=("gated", "plain"))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", MLP)
def test_mlp_variants(T, k, E, H, F, dtype, gated):
    """All tokens have an expert in common, so that it has as many rows at a time as there may be."""
    x, w1, t1, w2, t2, ids, weights = make(T + H, T, k, E, H, F, gated, dtype)
    ids[:, 0] = E // 2
    whole, y = guarded(T, H, dtype)
    amd.mxfp4_moe_mlp(x, t1, t2, ids, weights, y=y)
    check(y, x, w1, w2, ids, weights, E, gated)
    assert untouched(whole, T * H)


# --- what the order of the sums follows from ------------------------------------

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,K", [(100, 400), (300, 4096), (3000, 1000), (40, 20000)])
def test_gemv_row_does_not_know_the_others(N, K, dtype):
    """The order follows from the sizes and the type: other rows' values leave a row's bits alone."""
    _, wt = random_rows(N, N, K, 118, 130)
    g = torch.Generator(device=dev()).manual_seed(K)
    for M in (2, 5, 6, 9, 13, 14, 16):
        x = torch.randn(M, K, generator=g, device=dev()).to(dtype)
        y = amd.mxfp4_gemv(x, wt, out_dtype=F32)
        for row in (0, M - 1):
            other = torch.randn(M, K, generator=g, device=dev()).to(dtype)
            other[row] = x[row]
            assert bits(amd.mxfp4_gemv(other, wt, out_dtype=F32)[row], y[row]), (M, row)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", [(16, 4, 9, 100, 23), (20, 3, 5, 257, 41), (64, 2, 3, 600, 130), (3, 2, 8, 2048, 64)])
def test_mlp_token_does_not_know_the_others(T, k, E, H, F, dtype):
    """The same for a layer's tokens, where the ids stay."""
    x, w1, t1, w2, t2, ids, weights = make(T, T, k, E, H, F, True, dtype)
    y = amd.mxfp4_moe_mlp(x, t1, t2, ids, weights)
    for token in (0, T // 2, T - 1):
        other, scale = x.flip(0).contiguous(), weights.flip(0).contiguous()
        other[token], scale[token] = x[token], weights[token]
        assert bits(amd.mxfp4_moe_mlp(other, t1, t2, ids, scale)[token], y[token])


# --- the expert layer's rows between its products -----------------------------

# tokens, slots, experts, H, F: F off the 16 channels of a tile, and no expert's rows a whole tile of scales
ODD = [(1, 1, 1, 64, 1), (3, 2, 5, 130, 33), (5, 2, 3, 300, 70), (16, 4, 9, 100, 23), (20, 3, 5, 257, 41),
       (40, 2, 3, 64, 129), (2, 2, 3, 2500, 140), (64, 2, 3, 40, 17)]


@pytest.mark.parametrize("gated", (True, False), ids=("gated", "plain"))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", ODD)
def test_mlp_scales_of_rows_past_the_last(T, k, E, H, F, dtype, gated):
    x, w1, t1, w2, t2, ids, weights = make(T + F, T, k, E, H, F, gated, dtype)
    clean = amd.mxfp4_moe_mlp(x, t1, t2, ids, weights)
    assert clean.isfinite().all()
    for a, b in ((padded(t1), t2), (t1, padded(t2) if t2.rows % 32 else t2)):
        assert bits(amd.mxfp4_moe_mlp(x, a, b, ids, weights), clean)


@pytest.mark.parametrize("gated", (True, False), ids=("gated", "plain"))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", [c for c in ODD if c[2] > 1])
def test_mlp_nan_channel_of_the_next_expert(T, k, E, H, F, dtype, gated):
    """Its first channel stands behind this one's last in the same tile of scales."""
    x, w1, t1, w2, t2, ids, weights = make(T + F, T, k, E, H, F, gated, dtype)
    clean = amd.mxfp4_moe_mlp(x, t1, t2, ids, weights)
    codes, scales = t1.blocks()
    sick = E // 2
    scales[sick * F * (2 if gated else 1)] = 255
    y = amd.mxfp4_moe_mlp(x, amd.Mxfp4Tensor.from_blocks(codes, scales, H), t2, ids, weights)
    hit = (ids == sick).any(1)
    assert bits(y[~hit], clean[~hit]) and y[hit].isnan().all()


@pytest.mark.parametrize("gated", (True, False), ids=("gated", "plain"))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T", (1, 3, 20))
def test_mlp_infinite_weight_of_the_router(T, dtype, gated):
    """One channel between the products, positive: y is an infinity with the sign of W2's value.  (The
    channels past F, zeros, are not multiplied by the router's weight.)"""
    E, H = 2, 48
    x = torch.full((T, H), 0.5, dtype=dtype, device=dev())
    g = torch.Generator(device=dev()).manual_seed(T)
    one = torch.full((E * (2 if gated else 1), 2, 16), 0x22, dtype=torch.uint8, device=dev())      # ones
    t1 = amd.Mxfp4Tensor.from_blocks(one, torch.full(one.shape[:2], 127, dtype=torch.uint8, device=dev()), H)
    code = torch.randint(1, 8, (E * H, 1, 16), generator=g, device=dev(), dtype=torch.uint8)
    code |= torch.randint(0, 2, code.shape, generator=g, device=dev(), dtype=torch.uint8) << 3
    t2 = amd.Mxfp4Tensor.from_blocks(code, torch.full((E * H, 1), 127, dtype=torch.uint8, device=dev()), 1)
    ids = torch.arange(T, device=dev()).view(T, 1) % E
    y = amd.mxfp4_moe_mlp(x, t1, t2, ids, torch.full((T, 1), INF, device=dev()))
    want = t2.dequant(out_dtype=F32).view(E, H).sign()[ids[:, 0]] * INF
    assert same(y, want.to(dtype))


# --- rows sorted by expert in the largest tiles --------------------------------

# rows of each expert (the rest of the slots, two to a token, are dropped), slots, N, K; whether a turn's
# tiles are computed whole, and what becomes of the last turn's
LARGE = [((1400, 1300, 1396), 4096, 5000, 260, (True, "halves")), ((4096,), 4096, 4300, 130, (True, "quarters")),
         ((2000, 2096), 4096, 6100, 260, (True, "whole")), ((4096,), 4096, 8000, 300, (True, "whole")),
         ((0, 3000, 0, 1, 1095), 4096, 3800, 200, (True, "quarters")), ((1700, 0, 900), 4000, 6100, 520, (True, "quarters")),
         ((0, 1300, 500), 4096, 3800, 260, (False, "halves"))]


def shares(counts, N, cus):
    """Whether there are whole tiles of 256 x 256, and how the others are computed."""
    tiles = sum(-(-c // 256) for c in counts) * -(-N // 256)
    rest = tiles % cus if 2 * (tiles % cus) <= cus else 0
    return tiles > rest, "whole" if rest == 0 else "quarters" if 4 * rest <= cus else "halves"


@pytest.mark.parametrize("counts,slots,N,K,kind", LARGE)
def test_grouped_in_the_largest_tiles(counts, slots, N, K, kind):
    """Every share of a launch, in every type, with rows that have no source and channels that are NaN."""
    E, T = len(counts), slots // 2
    assert plan(slots, N, K, E)[0] == 5
    assert shares(counts, N, torch.cuda.get_device_properties(0).multi_processor_count) == kind
    ids = torch.full((slots,), -1)
    ids[:sum(counts)] = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    ids = ids[torch.randperm(slots, generator=torch.Generator().manual_seed(N))].view(T, 2)
    route = amd.moe_sort(ids.to(dev()), E)
    x, xt = random_rows(N, T, K, 127, 129)
    w, wt = random_rows(K, E * N, K, 127, 129)
    codes, scales = wt.blocks()
    scales[5::1000], w[5::1000] = 255, NAN
    wt = amd.Mxfp4Tensor.from_blocks(codes, scales, K)
    order = route.order.clone()
    order[3::5], order[4::11] = -1, slots + 9
    token = (order.long() // 2).clamp(0, T - 1)
    gone = (order < 0) | (order >= slots)
    offsets = route.offsets.tolist()
    for dtype in TYPES:
        for o, none in ((route.order, None), (order, gone)):
            whole, y = guarded(slots, N, dtype)
            amd.mxfp4_gemm_grouped(xt, wt, amd.MoeRoute(route.offsets, o, route.pos), y=y)
            assert untouched(whole, slots * N) and (y[offsets[E]:] == 7.25).all()
            for e in range(E):
                a, b = offsets[e], offsets[e + 1]
                rows = x[token[a:b]] if none is not None else x[(o[a:b].long() // 2)]
                we = w[e * N:(e + 1) * N]
                ok = ~we[:, 0].isnan()
                want = torch.full((b - a, N), NAN, dtype=dtype, device=dev())
                if a < b:
                    want[:, ok] = exactly(rows, we[ok], 0.25, dtype)
                if none is not None:
                    want[none[a:b]] = 0.0
                assert same(y[a:b], want), (dtype, e)


@pytest.mark.parametrize("T,k,E,N,K", [(8, 2, 4, 50, 300), (16, 4, 64, 900, 512), (208, 3, 5, 163, 190), (586, 4, 2, 3044, 260),
                                       (2048, 2, 3, 4400, 130)])
def test_grouped_offsets_are_clamped(T, k, E, N, K):
    """An end below zero and one past the rows: the first expert has none, the second's begin with row 0,
    and the last one's go on to the last row: behind the sorted ones, which have no slot and give zeros."""
    x, xt = random_rows(1, T, K, 127, 129)
    w, wt = random_rows(2, E * N, K, 127, 129)
    ids = torch.arange(T * k).view(T, k) % E
    ids[::7, 0] = -1
    route = amd.moe_sort(ids.to(dev()), E)
    wild = route.offsets.clone()
    wild[1], wild[-1] = -5, 1 << 30
    offsets = wild.clamp(0, T * k).tolist()
    for dtype in TYPES:
        whole, y = guarded(T * k, N, dtype)
        amd.mxfp4_gemm_grouped(xt, wt, amd.MoeRoute(wild, route.order, route.pos), y=y)
        assert untouched(whole, T * k * N)
        for e in range(1, E):
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                order = route.order[a:b].long()
                want = exactly(x[order.clamp(0) // k], w[e * N:(e + 1) * N], 0.25, dtype)
                want[order < 0] = 0.0
                assert same(y[a:b], want), (dtype, e)
