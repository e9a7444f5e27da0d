"""GPU parity of the expert layer of a few tokens (mxfp4_moe_mlp) with the
definition in 64 bits, and of the composed layer around mxfp4_gemm_grouped.

How far y may be off: W1 x is a sum of H exact products within v = terms * 2^-23 *
S of the exact one (S the sum of magnitudes, terms as in test_gpu_mxfp4.py); |silu'| <
1.1 and |silu(g)| <= |g|, so what lies between is off by 1.1 v |other| + |gate| v and the
products' errors of 2^-20 relative (exp, a division, two products), times the router's
weight, and is kept to 2^-17 (2^-24 for fp32) of itself.  The second product multiplies all
of that by |W2| and adds terms of its own; y is rounded once."""
import pytest
import torch

import w4a16_gemv_amd as amd
from tests.test_gpu_mxfp4 import BF, F32, TYPES, dev, guarded, random_rows, same, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def layer(x, w1, w2, ids, weights, E, gated):
    """(y, its bound before y's rounding), fp64."""
    T, H = x.shape
    F = w2.shape[1]
    x = x.double()
    y, off = torch.zeros(T, H, dtype=torch.float64, device=dev()), torch.zeros(T, H, dtype=torch.float64, device=dev())
    up = 2 * F if gated else F
    small = 2.0 ** -24 if x.dtype == F32 else 2.0 ** -17
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            a, b = w1[e * up:(e + 1) * up], w2[e * H:(e + 1) * H]
            p = 1.0 if weights is None else float(weights[t, j])
            v = a @ x[t]
            dv = (3 * H / 32 + 10) * 2.0 ** -23 * (a.abs() @ x[t].abs())
            gate, dgate = v[:F], dv[:F]
            s = gate * torch.sigmoid(gate)
            if gated:
                h = s * v[F:]
                dh = 1.1 * dgate * v[F:].abs() + s.abs() * dv[F:] + 1.1 * dgate * dv[F:]
            else:
                h, dh = s, 1.1 * dgate
            dh = dh + h.abs() * (2.0 ** -19 + small)
            y[t] += p * (b @ h)
            terms = 3 * F * ids.shape[1] / 32 + 3 * ids.shape[1] + 10
            off[t] += abs(p) * (b.abs() @ dh + terms * 2.0 ** -23 * (b.abs() @ (h.abs() + dh)))
    return y, off


def check(y, x, w1, w2, ids, weights, E, gated):
    want, off = layer(x, w1, w2, ids.cpu(), weights, E, gated)
    eps = torch.finfo(y.dtype).eps
    limit = off * (1 + eps) + want.abs() * eps / 2 + torch.finfo(y.dtype).tiny * eps
    worst = ((y.double() - want).abs() / limit).max()
    assert ((y.double() - want).abs() <= limit).all(), f"worst error / bound {float(worst):.3g}"


def make(seed, T, k, E, H, F, gated, dtype, drop=0.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    w1, t1 = random_rows(seed, E * F * (2 if gated else 1), H, 118, 122)
    w2, t2 = random_rows(seed + 1, E * H, F, 118, 122)
    x = torch.randn(T, H, generator=g, device=dev()).to(dtype)
    ids = torch.rand(T, E, generator=g, device=dev()).topk(min(k, E), 1).indices if k <= E else \
        torch.randint(0, E, (T, k), generator=g, device=dev())
    if drop:
        ids[torch.rand(ids.shape, generator=g, device=dev()) < drop] = -1
    weights = torch.rand(ids.shape, generator=g, device=dev())
    return x, w1, t1, w2, t2, ids, weights


CASES = [(1, 1, 1, 16, 16), (1, 2, 8, 512, 256), (2, 1, 2, 33, 1), (3, 4, 64, 101, 33), (4, 2, 4, 300, 129),
         (5, 2, 3, 1001, 333), (8, 3, 16, 130, 640), (9, 2, 4, 17, 70), (16, 4, 64, 256, 128), (17, 4, 8, 64, 96),
         (33, 2, 5, 100, 60), (64, 8, 128, 48, 40), (64, 2, 1, 40, 300), (40, 6, 200, 20, 20), (1, 32, 1024, 64, 32),
         (13, 8, 1024, 16, 24), (2, 2, 3, 2500, 140)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", CASES)
def test_mlp(T, k, E, H, F, dtype):
    for gated in (True, False):
        x, w1, t1, w2, t2, ids, weights = make(T + F, T, k, E, H, F, gated, dtype, drop=0.1 if T > 1 else 0.0)
        for i, w in ((ids, weights), (ids.int(), None)):
            whole, y = guarded(T, H, dtype)
            assert amd.mxfp4_moe_mlp(x, t1, t2, i, w, y=y) is y
            check(y, x, w1, w2, i, w, E, gated)
            assert untouched(whole, T * H)


@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 4, 4096, 1500), (7, 2, 3, 1024, 2050), (20, 3, 6, 700, 900), (16, 4, 64, 256, 600),
                                       (16, 4, 64, 900, 600), (9, 4, 64, 2000, 600),
                                       (4, 2, 8, 2500, 300), (16, 4, 64, 2050, 130)])
def test_mlp_larger(T, k, E, H, F):
    x, w1, t1, w2, t2, ids, weights = make(2, T, k, E, H, F, True, BF)
    check(amd.mxfp4_moe_mlp(x, t1, t2, ids, weights), x, w1, w2, ids, weights, E, True)


def test_mlp_slots_of_one_expert_and_none():
    """All tokens to one expert; the same expert twice in a token; tokens without a slot give zeros."""
    T, k, E, H, F = 20, 3, 5, 100, 70
    x, w1, t1, w2, t2, ids, weights = make(3, T, k, E, H, F, True, F32)
    for change in ("one", "twice", "none", "all dropped"):
        i = ids.clone()
        if change == "one":
            i[:] = 2
        elif change == "twice":
            i[:, 1] = i[:, 0]
        elif change == "none":
            i[3:9], i[12, 1] = -1, 1 << 40
        else:
            i[:] = E
        y = amd.mxfp4_moe_mlp(x, t1, t2, i, weights, y=torch.full((T, H), 7.0, device=dev()))
        check(y, x, w1, w2, i, weights, E, True)
        assert not y[((i < 0) | (i >= E)).all(1)].any()


def test_mlp_nan_stays_where_it_belongs():
    """A channel of an expert that is NaN, a token that is, and unused columns beside them."""
    T, k, E, H, F = 9, 2, 6, 80, 50
    x, w1, t1, w2, t2, ids, weights = make(4, T, k, E, H, F, True, BF)
    clean = amd.mxfp4_moe_mlp(x, t1, t2, ids, weights)
    codes, scales = t2.blocks()
    scales[3 * H + 11, 1] = 255       # channel 11 of expert 3's way down
    hurt = amd.Mxfp4Tensor.from_blocks(codes, scales, F)
    x2 = x.clone()
    x2[4, 7] = float("inf")
    y = amd.mxfp4_moe_mlp(x2, t1, hurt, ids, weights)
    want = clean.clone()
    want[(ids == 3).any(1), 11] = float("nan")
    rest = [t for t in range(T) if t != 4]
    assert same(y[rest], want[rest]) and not y[4].isfinite().all()


def test_mlp_empty():
    x, w1, t1, w2, t2, ids, weights = make(5, 4, 2, 3, 64, 32, True, BF)
    assert amd.mxfp4_moe_mlp(x[:0], t1, t2, ids[:0], weights[:0]).shape == (0, 64)
    none = amd.Mxfp4Tensor(torch.zeros(3 * 64, 0, dtype=torch.uint8, device=dev()),
                           torch.zeros(0, dtype=torch.uint8, device=dev()), 0)
    w = amd.Mxfp4Tensor(torch.zeros(0, 64, dtype=torch.uint8, device=dev()),
                        torch.zeros(0, dtype=torch.uint8, device=dev()), 64)
    y = torch.full((4, 64), 7.0, dtype=BF, device=dev())
    assert not amd.mxfp4_moe_mlp(x, w, none, ids, weights, y=y).any()


def test_mlp_refusals():
    x, w1, t1, w2, t2, ids, weights = make(6, 4, 2, 3, 64, 32, True, BF)
    _, narrow = random_rows(7, 3 * 64, 20)
    f = amd.mxfp4_moe_mlp
    for bad, match in (((x[0], t1, t2, ids, weights), "x must be"), ((x, t2, t2, ids, weights), "w1 has K=32"),
                       ((x, t1, narrow, ids, weights), "w1 has 192 rows"), ((x, t1, t2, ids[:3], weights), "ids must be"),
                       ((x, t1, t2, ids.float(), weights), "int32 or int64"), ((x, t1, t2, ids, weights.half()), "weights must be"),
                       ((x, t1, t2, ids, weights[:, :1]), "weights must be"), ((x, t1, t2, ids.t().contiguous().t(), weights), "contiguous"),
                       ((x, t1, t2, ids.cpu(), weights), "ids is on")):
        with pytest.raises(ValueError, match=match):
            f(*bad)
    with pytest.raises(ValueError, match="at most 64 tokens"):
        f(x[:1].repeat(65, 1), t1, t2, ids[:1].repeat(65, 1))
    with pytest.raises(ValueError, match="at most 64 tokens"):
        f(x, t1, t2, ids[:, :1].repeat(1, 33))
    with pytest.raises(ValueError, match="y must be"):
        f(x, t1, t2, ids, weights, y=torch.empty(4, 64, device=dev()))
    with pytest.raises(ValueError, match="requires a gradient"):
        f(x, t1, t2, ids, weights.clone().requires_grad_())
    with pytest.raises(amd.NF4Error):
        f(x, t1, t2, ids, weights, workspace=torch.empty(256, dtype=torch.uint8, device=dev()))


@pytest.mark.parametrize("T", [1, 16, 50])
def test_mlp_graphs(T):
    """Two captured layers one after the other, replayed with other tokens and other routings."""
    k, E, H, F = 2, 16, 512, 300
    x, w1, t1, w2, t2, ids, weights = make(7, T, k, E, H, F, True, BF)
    amd.mxfp4_moe_mlp(x, t1, t2, ids, weights)
    out = [torch.empty_like(x) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        amd.mxfp4_moe_mlp(x, t1, t2, ids, weights, y=out[0])
        amd.mxfp4_moe_mlp(out[0], t1, t2, ids, weights, y=out[1])
    g = torch.Generator(device=dev()).manual_seed(8)
    for turn in range(4):
        x.copy_(torch.randn(T, H, generator=g, device=dev()))
        ids.copy_(torch.randint(-1, E, (T, k), generator=g, device=dev()))
        weights.copy_(torch.rand(T, k, generator=g, device=dev()))
        for o in out:
            o.fill_(-1.0)
        graph.replay()
        first = amd.mxfp4_moe_mlp(x, t1, t2, ids, weights)
        assert torch.equal(out[0], first) and torch.equal(out[1], amd.mxfp4_moe_mlp(first, t1, t2, ids, weights))
        torch.cuda.synchronize()


def test_the_composed_layer():
    """moe_sort, the quantized products, moe_combine: what a prompt takes, next to the layer of few tokens.

    By definition with the codes of x and of what lies between taken from the encoder, whose own
    tests are exact: so only fp32 sums and the roundings to fp32 differ."""
    T, k, E, H, F = 50, 3, 6, 256, 200
    x, w1, t1, w2, t2, ids, weights = make(9, T, k, E, H, F, True, F32)
    route = amd.moe_sort(ids, E)
    v = amd.mxfp4_gemm_grouped(amd.mxfp4_quantize(x), t1, route, out_dtype=F32)
    h = torch.nn.functional.silu(v[:, :F]) * v[:, F:]
    hq = amd.mxfp4_quantize(h)
    o = amd.mxfp4_gemm_grouped(hq, t2, route, out_dtype=F32, x_sorted=True)
    y = amd.moe_combine(o, route, weights)
    xq = amd.mxfp4_quantize(x).dequant(out_dtype=F32).double()
    hv = hq.dequant(out_dtype=F32).double()
    order = route.order.long().cpu()
    want, S = torch.zeros(T, H, dtype=torch.float64, device=dev()), torch.zeros(T, H, dtype=torch.float64, device=dev())
    for i, slot in enumerate(order.tolist()):
        t, e = slot // k, int(ids.view(-1)[slot])
        exact = w1[e * 2 * F:(e + 1) * 2 * F] @ xq[t]
        limit = (H / 64 + 17) * 2.0 ** -23 * (w1[e * 2 * F:(e + 1) * 2 * F].abs() @ xq[t].abs())
        assert ((v[i].double() - exact).abs() <= limit + 2.0 ** -24 * exact.abs()).all()
        p = float(weights.view(-1)[slot])
        want[t] += p * (w2[e * H:(e + 1) * H] @ hv[i])
        S[t] += p * (w2[e * H:(e + 1) * H].abs() @ hv[i].abs())
    assert ((y.double() - want).abs() <= (F / 64 + 17 + k + 2) * 2.0 ** -23 * S).all()
    # the layer of few tokens keeps the activations' bits: it is nearer to the exact layer
    true, off = layer(x, w1, w2, ids.cpu(), weights, E, True)
    few = amd.mxfp4_moe_mlp(x, t1, t2, ids, weights).double()
    assert (few - true).norm() < 0.01 * (y.double() - true).norm()


def test_mlp_offsets_past_4_gib():
    """Experts whose codes lie past 4 GiB of both matrices."""
    T, H, F, E = 2, 2048, 4096, 1024
    rows1, rows2 = E * F, E * H
    d1 = torch.zeros((rows1, amd.mxfp4_pitch(H)), dtype=torch.uint8, device=dev())
    d2 = torch.zeros((rows2, amd.mxfp4_pitch(F)), dtype=torch.uint8, device=dev())
    s1 = torch.full((amd.mxfp4_scale_size(rows1, H),), 120, dtype=torch.uint8, device=dev())
    s2 = torch.full((amd.mxfp4_scale_size(rows2, F),), 120, dtype=torch.uint8, device=dev())
    assert d1.numel() >= 1 << 32 and d2.numel() >= 1 << 32
    w1, t1 = random_rows(1, F, H, 120, 121)
    w2, t2 = random_rows(2, H, F, 120, 121)
    d1[-F:], d2[-H:] = t1.data, t2.data
    x = torch.randn(T, H, generator=torch.Generator(device=dev()).manual_seed(1), device=dev()).to(BF)
    ids = torch.tensor([[E - 1, 5], [700, E - 1]], device=dev())
    big1, big2 = amd.Mxfp4Tensor(d1, s1, H), amd.Mxfp4Tensor(d2, s2, F)
    y = amd.mxfp4_moe_mlp(x, big1, big2, ids)
    check(y, x, w1, w2, torch.zeros(2, 1, dtype=torch.int64), None, 1, False)
