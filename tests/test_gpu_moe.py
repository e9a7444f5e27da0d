"""GPU parity of the expert routing (include/moe.h) against the definitions:
whole numbers and moved rows are compared exactly, sums within bounds that
follow from the number of fp32 roundings."""
import numpy as np
import pytest
import torch

import w4a16_gemv_amd as amd
from tests.test_gpu_int8 import (BF, F32, FP, TYPES, dev, encode, guarded, product, random_tensor, route_of, same,
                                 to_route, untouched)

pytestmark = pytest.mark.gpu

HALF_STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -134, FP: 2.0 ** -25, F32: 2.0 ** -150}     # half a step among the subnormals


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


def random_ids(rng, T, k, E, kind, dtype=np.int64):
    ids = rng.integers(0, max(E, 1), (T, k))
    if kind == "drop":
        ids[rng.random((T, k)) < 0.25] = -1
        ids[rng.random((T, k)) < 0.1] = E
        ids[: T // 5] = -7
    elif kind == "none":
        ids[:] = -1
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "far":
        ids[rng.random((T, k)) < 0.5] = np.iinfo(dtype).max if dtype == np.int64 else 2 ** 31 - 1
        ids[rng.random((T, k)) < 0.2] = np.iinfo(dtype).min
    return ids.astype(dtype)


SORTS = [(1, 1, 1, "all"), (1, 2, 8, "all"), (0, 2, 8, "all"), (16, 4, 64, "all"), (63, 1, 3, "drop"), (64, 1, 2, "all"),
         (65, 1, 1, "all"), (128, 8, 1024, "all"), (100, 3, 7, "far"), (50, 2, 9, "none"), (511, 2, 5, "one"), (1000, 4, 64, "drop"),
         (1024, 4, 16, "all"), (1025, 4, 16, "all"), (4097, 1, 33, "drop"), (8191, 4, 64, "drop"), (3000, 8, 1024, "all"),
         (20000, 2, 1, "all"), (30000, 3, 100, "one"), (9000, 1, 6, "none"), (5000, 2, 0, "all"), (4, 2, 0, "all"),
         (300000, 4, 128, "drop"), (1024, 1, 16, "drop"), (1025, 1, 16, "drop"), (512, 4, 1024, "drop"), (2049, 1, 40, "far"),
         (4096, 1, 7, "drop"), (2049, 2, 64, "drop"), (8192, 4, 64, "drop"), (32769, 1, 12, "far"), (16383, 2, 1024, "all")]


@pytest.mark.parametrize("T,k,E,kind", SORTS)
@pytest.mark.parametrize("dtype", [np.int32, np.int64])
def test_sort(T, k, E, kind, dtype):
    rng = np.random.default_rng(T + k + E)
    ids = random_ids(rng, T, k, E, kind, dtype)
    flat = ids.reshape(-1).astype(np.int64)
    kept = (flat >= 0) & (flat < E)
    rows = np.argsort(np.where(kept, flat, E), kind="stable")[:kept.sum()]
    order = np.full(T * k, -1, np.int32)
    order[:rows.size] = rows
    pos = np.full(T * k, -1, np.int32)
    pos[rows] = np.arange(rows.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))]).astype(np.int32)[:E + 1]
    for _ in range(2):
        r = amd.moe_sort(torch.from_numpy(ids).to(dev()), E)
        assert (r.T, r.top_k, r.rows, r.experts) == (T, k, T * k, E)
        assert np.array_equal(r.offsets.cpu().numpy(), offsets)
        assert np.array_equal(r.order.cpu().numpy(), order)
        assert np.array_equal(r.pos.cpu().numpy(), pos.reshape(T, k))


def test_sort_workspace():
    ids = torch.randint(0, 9, (4000, 4), device=dev())
    want = amd.moe_sort(ids, 9)
    work = torch.full((amd.load().moe_sort_workspace_size(4000, 4, 9),), 255, dtype=torch.uint8, device=dev())
    for _ in range(2):
        got = amd.moe_sort(ids, 9, workspace=work)
        for name in ("offsets", "order", "pos"):
            assert torch.equal(getattr(got, name), getattr(want, name))
    with pytest.raises(amd.NF4Error):
        amd.moe_sort(ids, 9, workspace=work[:-1].contiguous()[:256])
    with pytest.raises(amd.NF4Error) as e:
        amd.moe_sort(ids, 1025)
    assert e.value.status == amd.NF4_EUNSUPPORTED


MOVES = [(1, 1, 1, 1, "all"), (1, 2, 8, 4096, "all"), (16, 4, 64, 2048, "all"), (5, 3, 4, 7, "drop"), (33, 2, 3, 8, "all"),
         (20, 8, 16, 129, "drop"), (64, 1, 5, 1001, "one"), (9, 2, 4, 2049, "drop"), (7, 5, 6, 8200, "all"),
         (10, 2, 3, 300, "none"), (0, 2, 3, 64, "all"), (6, 2, 3, 0, "all"), (300, 4, 8, 513, "drop"), (3, 12, 20, 264, "all"),
         (4, 40, 50, 72, "drop"), (50, 3, 4, 1023, "all"),
         (7, 5, 8, 1024, "drop"), (9, 2, 4, 1025, "drop"), (2049, 2, 4, 520, "drop")]


def problem(T, k, E, kind, seed):
    rng = np.random.default_rng(seed)
    ids = random_ids(rng, T, k, E, kind)
    offsets, order, pos = route_of(ids, E)
    weights = rng.uniform(-0.5, 1.5, (T, k)).astype(np.float32)
    return rng, pos, to_route((offsets, order, pos)), weights


def shifted(t, shift):
    """A GPU copy of t that starts `shift` elements into its allocation."""
    room = torch.zeros(t.numel() + shift, dtype=t.dtype, device=dev())
    v = room[shift:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,kind", MOVES)
def test_gather(T, k, E, H, kind, dtype):
    rng, pos, plan, _ = problem(T, k, E, kind, T + H)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype)
    want = torch.full((T * k, H), 7.25, dtype=dtype)
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[pos[t, j]] = x[t]
    for shift in (0, 1):
        whole, xs = guarded(T * k, H, dtype)
        assert amd.moe_gather(shifted(x, shift), plan, out=xs) is xs
        assert same(xs, want) and untouched(whole, T * k * H)


def sums(pos, weights, ys):
    """(sum_j w ys, sum_j |w ys|) per token in 64 bits."""
    T, k = pos.shape
    v, s = np.zeros((T, ys.shape[1])), np.zeros((T, ys.shape[1]))
    for j in range(k):
        on = pos[:, j] >= 0
        term = weights[on, j, None].astype(np.float64) * ys[pos[on, j]]
        v[on] += term
        s[on] += np.abs(term)
    return v, s


def close(got, v, s, roundings, dtype):
    """Within `roundings` fp32 roundings of sums of magnitude s, and one to dtype."""
    got = got.double().cpu().numpy()
    band = roundings * 2.0 ** -24 * s * (1 + 2.0 ** -12)
    ok = np.abs(got - v) <= band + HALF_STEP[dtype] * (np.abs(v) + band) + TINY[dtype]
    return bool(ok.all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,kind", MOVES)
def test_combine(T, k, E, H, kind, dtype):
    rng, pos, plan, weights = problem(T, k, E, kind, 2 * T + H)
    ys = torch.from_numpy(rng.standard_normal((T * k, H))).to(dtype)
    live = np.zeros(T * k, bool)
    live[pos[pos >= 0]] = True
    ys[torch.from_numpy(~live)] = float("nan")              # rows that no slot has are never read
    wt = torch.from_numpy(weights).to(dev())
    v, s = sums(pos, weights, np.nan_to_num(ys.double().numpy()))
    ones_v, ones_s = sums(pos, np.ones_like(weights), np.nan_to_num(ys.double().numpy()))
    for shift in (0, 1):
        whole, y = guarded(T, H, dtype)
        assert amd.moe_combine(shifted(ys, shift), plan, wt, out=y) is y
        assert close(y, v, s, k, dtype) and untouched(whole, T * H)
        y = amd.moe_gather_grad(shifted(ys, shift), plan)
        assert close(y, ones_v, ones_s, k, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,kind", MOVES)
def test_combine_grad(T, k, E, H, kind, dtype):
    rng, pos, plan, weights = problem(T, k, E, kind, 3 * T + H)
    ys = torch.from_numpy(rng.standard_normal((T * k, H))).to(dtype)
    dy = torch.from_numpy(rng.standard_normal((T, H))).to(dtype)
    wt = torch.from_numpy(weights).to(dev())
    for w in (wt, None):
        wv = weights if w is not None else np.ones_like(weights)
        want = torch.full((T * k, H), 7.25, dtype=dtype)
        for t in range(T):
            for j in range(k):
                if pos[t, j] >= 0:  # one fp32 product, rounded once
                    want[pos[t, j]] = torch.from_numpy(wv[t, j] * dy[t].float().numpy()).to(dtype)
        at = np.maximum(pos, 0)
        terms = ys.double().numpy()[at] * dy.double().numpy()[:, None, :] if T * k else np.zeros((T, k, H))
        terms *= (pos >= 0)[..., None]
        for shift in (0, 1):
            whole, dys = guarded(T * k, H, dtype)
            got, dw = amd.moe_combine_grad(shifted(dy, shift), shifted(ys, shift), plan, w, dys=dys)
            assert got is dys and same(dys, want) and untouched(whole, T * k * H)
            # a lane's chain is at most H / 64 long and rounded up to a piece; the rest is a tree
            assert close(dw, terms.sum(-1), np.abs(terms).sum(-1), H / 64 + 24, F32)
            assert bool((dw.cpu()[torch.from_numpy(pos < 0)] == 0).all())


def test_combine_grad_parts_through_the_c_abi():
    """Either result alone; ys is not read without dweights."""
    _, pos, plan, weights = problem(30, 2, 4, "drop", 8)
    H = 100
    ys, dy = torch.randn(60, H, device=dev()), torch.randn(30, H, device=dev())
    wt = torch.from_numpy(weights).to(dev())
    dys, dw = amd.moe_combine_grad(dy, ys, plan, wt, dys=torch.zeros(60, H, device=dev()))
    a, b = torch.zeros(60, H, device=dev()), torch.full((30, 2), 9.0, device=dev())
    f, st = amd.load().moe_combine_grad, torch.cuda.current_stream().cuda_stream
    args = (2, wt.data_ptr(), plan.pos.data_ptr(), 30, 2, 60, H)
    assert f(dy.data_ptr(), None, *args, a.data_ptr(), None, st) == 0
    assert f(dy.data_ptr(), ys.data_ptr(), *args, None, b.data_ptr(), st) == 0
    assert same(a, dys) and same(b, dw)


def test_gradients_against_differences():
    """Combine is linear in ys and in the weights, so a difference of two outputs is the gradient's
    product with the step; with small whole numbers every fp32 operation is exact and so are they."""
    rng, pos, plan, _ = problem(40, 3, 5, "drop", 21)
    H = 200
    whole = lambda *shape: torch.from_numpy(rng.integers(-8, 9, shape)).float().to(dev())  # noqa: E731
    ys, step, dy = whole(120, H), whole(120, H), whole(40, H)
    w, dstep = whole(40, 3) / 4, whole(40, 3) / 4
    dys, dw = amd.moe_combine_grad(dy, ys, plan, w, dys=torch.zeros(120, H, device=dev()))
    base = amd.moe_combine(ys, plan, w)
    inner = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    assert inner(dys, step) == inner(dy, amd.moe_combine(ys + step, plan, w) - base)
    assert inner(dw, dstep) == inner(dy, amd.moe_combine(ys, plan, w + dstep) - base)
    x, xstep, g = whole(40, H), whole(40, H), whole(120, H)
    zero = lambda: torch.zeros(120, H, device=dev())  # noqa: E731
    moved = amd.moe_gather(x + xstep, plan, out=zero()) - amd.moe_gather(x, plan, out=zero())
    assert inner(amd.moe_gather_grad(g, plan), xstep) == inner(g, moved)


def test_offsets_past_32_bits():
    """Rows beyond the first 4 GiB of their tensors."""
    T, H = 50000, 48001
    ids = torch.zeros(T, 1, dtype=torch.int32, device=dev())
    plan = amd.moe_sort(ids, 1)
    x = torch.empty(T, H, dtype=BF, device=dev())
    part = torch.randn(500, H, device=dev()).to(BF)
    for i in range(0, T, 500):
        x[i:i + 500] = part.roll(i // 500, 0)
    xs = amd.moe_gather(x, plan)
    assert torch.equal(xs, x)                                   # one expert, one slot: the same order
    assert torch.equal(amd.moe_gather_grad(xs, plan), x)
    w = torch.full((T, 1), 2.0, device=dev())
    dys, dw = amd.moe_combine_grad(x, xs, plan, w, dys=xs.clone())
    assert torch.equal(dys[-5:], x[-5:] * 2) and torch.equal(dys[:5], x[:5] * 2)
    v = x[-5:].double().cpu().numpy() ** 2
    assert close(dw[-5:, 0], v.sum(1), v.sum(1), H / 64 + 24, F32)


def test_positions_out_of_range_are_dropped():
    T, k, H = 6, 2, 70
    pos = np.arange(T * k, dtype=np.int32).reshape(T, k)
    bad = pos.copy()
    bad[0, 0], bad[1, 1], bad[2, 0], bad[3, 0] = T * k, -1, 2 ** 31 - 1, -2 ** 31
    drop = pos.copy()
    drop[(bad < 0) | (bad >= T * k)] = -1
    order, offsets = np.arange(T * k, dtype=np.int32), np.array([0, T * k], np.int32)
    a, b = to_route((offsets, order, bad)), to_route((offsets, order, drop))
    x, ys = torch.randn(T, H, device=dev()), torch.randn(T * k, H, device=dev())
    out = lambda: torch.zeros(T * k, H, device=dev())  # noqa: E731
    assert same(amd.moe_gather(x, a, out=out()), amd.moe_gather(x, b, out=out()))
    assert same(amd.moe_combine(ys, a), amd.moe_combine(ys, b))
    for u, v in zip(amd.moe_combine_grad(x, ys, a, dys=out()), amd.moe_combine_grad(x, ys, b, dys=out())):
        assert same(u, v)


def test_infinities_reach_only_their_token():
    _, pos, plan, weights = problem(12, 2, 3, "all", 4)
    ys = torch.randn(24, 90, device=dev())
    ys[int(pos[5, 0]), 3] = float("inf")
    ys[int(pos[7, 1]), 8] = float("nan")
    y = amd.moe_combine(ys, plan, torch.from_numpy(weights).to(dev())).cpu()
    assert (~torch.isfinite(y)).nonzero().tolist() == [[5, 3], [7, 8]]


def test_refusals():
    _, pos, plan, weights = problem(4, 2, 3, "all", 4)
    x, ys, wt = torch.randn(4, 8, device=dev()), torch.randn(8, 8, device=dev()), torch.from_numpy(weights).to(dev())
    for call in (lambda: amd.moe_gather(ys, plan), lambda: amd.moe_combine(x, plan, wt),
                 lambda: amd.moe_combine(ys, plan, wt[:, :1]), lambda: amd.moe_combine(ys, plan, wt.double()),
                 lambda: amd.moe_gather(x, plan, out=ys.half()), lambda: amd.moe_gather(x.double(), plan),
                 lambda: amd.moe_combine_grad(x, ys.half(), plan, wt), lambda: amd.moe_combine_grad(ys, ys, plan, wt),
                 lambda: amd.moe_gather(x.t().contiguous().t(), plan), lambda: amd.moe_combine(ys, plan, wt.cpu()),
                 lambda: amd.MoeRoute(plan.offsets, plan.order[:-1], plan.pos),
                 lambda: amd.MoeRoute(plan.offsets.long(), plan.order, plan.pos)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda t: amd.moe_gather(t, plan), lambda t: amd.moe_combine_grad(t, ys, plan, wt)):
        leaf = x.clone().requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call(leaf)
        with torch.no_grad():
            call(leaf)


# --- a layer of experts, as it is used ---------------------------------------

@pytest.mark.parametrize("T,k,E,H,F,drop", [(1, 2, 8, 256, 512, False), (24, 4, 16, 320, 200, False), (300, 2, 5, 192, 333, True)])
def test_layer_of_experts(T, k, E, H, F, drop):
    """Routing, two expert products with an activation between them, and the way back.  Every stage is
    checked by definition from what the stage before gave."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF).to(dev())
    ids = random_ids(rng, T, k, E, "drop" if drop else "all")
    wts = rng.uniform(0, 1, (T, k)).astype(np.float32)
    up, ups, upt = random_tensor(rng, E * F, H)
    down, downs, downt = random_tensor(rng, E * H, F)

    def layer():
        plan = amd.moe_sort(torch.from_numpy(ids).to(dev()), E)
        xq = amd.int8_quantize(x)
        h = amd.int8_gemm_grouped(xq, upt, plan, y=torch.zeros(T * k, F, dtype=BF, device=dev()))
        a = torch.relu(h)
        y = amd.int8_gemm_grouped(amd.int8_quantize(a), downt, plan, x_sorted=True,
                                  y=torch.zeros(T * k, H, dtype=BF, device=dev()))
        return h, a, y, amd.moe_combine(y, plan, torch.from_numpy(wts).to(dev()))

    h, a, y, out = layer()
    offsets, order, pos = route_of(ids, E)

    def experts(q, s, w, ws, N, src):
        want = torch.zeros(T * k, N, dtype=BF)
        for e in range(E):
            i, j = offsets[e], offsets[e + 1]
            if i < j:
                want[i:j] = product(q[src[i:j]], s[src[i:j]], w[e * N:(e + 1) * N], ws[e * N:(e + 1) * N], BF)
        return want

    q, s = encode(x.cpu())
    assert same(h, experts(q, s, up, ups, F, order // k))
    q, s = encode(a.cpu())
    assert same(y, experts(q, s, down, downs, H, np.arange(T * k)))
    v, m = sums(pos, wts, y.double().cpu().numpy())
    assert close(out, v, m, k, BF)
    # the activations gathered first give the same products
    plan = to_route((offsets, order, pos))
    xs = amd.moe_gather(x, plan, out=torch.zeros(T * k, H, dtype=BF, device=dev()))
    again = amd.int8_gemm_grouped(amd.int8_quantize(xs), upt, plan, x_sorted=True,
                                  y=torch.zeros(T * k, F, dtype=BF, device=dev()))
    assert same(again, h)


def test_training_step_in_an_autograd_function():
    """Gather and combine with their gradient functions inside torch.autograd.Function, against the same
    layer in fp64: every value is a small whole number, so fp32 is exact."""
    rng, pos, plan, _ = problem(20, 2, 4, "drop", 31)
    H = 48

    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return amd.moe_gather(x, plan, out=torch.zeros(plan.rows, H, device=dev()))

        @staticmethod
        def backward(ctx, g):
            return amd.moe_gather_grad(g.contiguous(), plan)

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ys, w):
            ctx.save_for_backward(ys, w)
            return amd.moe_combine(ys, plan, w)

        @staticmethod
        def backward(ctx, g):
            ys, w = ctx.saved_tensors
            return amd.moe_combine_grad(g.contiguous(), ys, plan, w, dys=torch.zeros_like(ys))

    whole = lambda *shape: torch.from_numpy(rng.integers(-4, 5, shape)).float().to(dev())  # noqa: E731
    x, w, c = whole(20, H).requires_grad_(), whole(20, 2).requires_grad_(), whole(20, H)
    y = Combine.apply(Gather.apply(x) * 3.0, w)
    (y * c).sum().backward()
    kept = torch.from_numpy(pos >= 0).to(dev()).double()
    x2, w2 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    y2 = ((w2 * kept)[..., None] * 3.0 * x2[:, None, :]).sum(1)
    (y2 * c.double()).sum().backward()
    assert torch.equal(y.double(), y2)
    assert torch.equal(x.grad.double(), x2.grad) and torch.equal(w.grad.double(), w2.grad)


def test_captured_and_replayed():
    T, k, E, H, N = 50, 2, 6, 130, 90
    rng = np.random.default_rng(17)
    w, ws, wt = random_tensor(rng, E * N, H)
    ids = torch.zeros(T, k, dtype=torch.int64, device=dev())
    big = torch.zeros(9000, 1, dtype=torch.int32, device=dev())
    x, wts = torch.zeros(T, H, device=dev()), torch.ones(T, k, device=dev())

    def layer():
        plan = amd.moe_sort(ids, E)
        ys = amd.int8_gemm_grouped(amd.int8_quantize(x), wt, plan, out_dtype=F32)
        y = amd.moe_combine(ys, plan, wts)
        dys, dw = amd.moe_combine_grad(y, ys, plan, wts)
        return plan.order, plan.pos, ys, y, dys, dw, amd.moe_sort(big, 40).order

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for _ in range(4):
        ids.random_(0, E), big.random_(-2, 40), x.normal_(), wts.uniform_()
        want = layer()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    rng = np.random.default_rng(18)
    jobs = []
    for T, k, E, H in ((7, 2, 8, 300), (3000, 4, 16, 65), (2000, 3, 700, 40), (500, 1, 3, 1001)):
        jobs.append((torch.from_numpy(random_ids(rng, T, k, E, "drop")).to(dev()), E, torch.randn(T, H, device=dev())))

    def job(ids, E, x):
        plan = amd.moe_sort(ids, E)
        xs = amd.moe_gather(x, plan, out=torch.zeros(plan.rows, x.shape[1], device=dev()))
        return plan.pos, xs, amd.moe_combine(xs, plan)

    want = [job(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(job(*j))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
