"""The operators of the int8 products and of expert routing as measurable cases.

Each case is one pass through one operator, in two forms: the plain form in elementary torch operations (`own`
false) and the calls a user makes of w4a16_gemv_amd (`own` true).  `exact` computes the same outputs in 64 bits
from the definitions.

Operators (the case's "op"):
  quantize     rows to int8 codes with one fp32 scale per row, and back to the values that the codes stand for:
               a = max(max|x|, 2^-100), scale = a / 127 and inverse = 127 / a in fp32, code = x * inverse rounded
               half to even, value = code * scale.
  linear       activations quantized per token on the way into the product with int8 weights that have a scale
               per output channel.
  gemm         the same product from activations that are quantized already.
  experts      the product for rows sorted by expert, each expert with weights of its own; the activations are
               read in token order through the routing's order.
  route        token slots sorted by expert, the tokens' rows gathered into that order, and the experts' outputs
               combined back per token with the router's weights.
  route_grad   the gradients of combine (to the experts' outputs and the router's weights) and of gather.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
FLOOR = 2.0 ** -100      # least maximum of a row that its scale is made from


def listed():
    return [
        # one decode step's token ahead of a projection
        dict(name="quantize_token", op="quantize", M=1, K=4096, x="bf16"),
        # the inner activation of an MLP over a long prompt, an odd number of rows
        dict(name="quantize_prompt", op="quantize", M=4097, K=11008, x="bf16"),
        # single-token decode of an attention projection
        dict(name="linear_token", op="linear", M=1, N=4096, K=4096, x="bf16", y="bf16"),
        # a small serving batch through an MLP projection
        dict(name="linear_batch", op="linear", M=13, N=11008, K=4096, x="fp16", y="fp16"),
        # sizes that no tile divides, everything in fp32
        dict(name="linear_ragged", op="linear", M=333, N=4099, K=1501, x="fp32", y="fp32"),
        # a long prompt through an MLP projection, quantized once for gate and up
        dict(name="gemm_prompt", op="gemm", M=8192, N=11008, K=4096, y="bf16"),
        # a decode step of 16 sequences over many small experts: few rows each, most experts' weights read
        dict(name="experts_token", op="experts", T=16, k=4, E=64, N=1024, K=2048, y="bf16", drop=0.0),
        # a prompt over a few large experts with uneven loads
        dict(name="experts_prompt", op="experts", T=4096, k=2, E=8, N=4096, K=4096, y="bf16", drop=0.0),
        # routing of the same decode step
        dict(name="route_token", op="route", T=16, k=4, E=64, H=2048, x="bf16", drop=0.0),
        # routing of a prompt, an odd number of tokens, padding tokens and slots of other ranks' experts dropped
        dict(name="route_prompt", op="route", T=8191, k=4, E=64, H=4096, x="bf16", drop=0.1),
        # a small training batch with an odd row width in fp32
        dict(name="route_grad_small", op="route_grad", T=257, k=2, E=8, H=1001, x="fp32", drop=0.0),
        # a training batch
        dict(name="route_grad_batch", op="route_grad", T=8192, k=4, E=64, H=4096, x="bf16", drop=0.0),
    ]


def _between(rng, lo, hi):
    """A whole number, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "gemm", "experts", "route", "route_grad"])
    x, y = rng.choice(sorted(DT)), rng.choice(sorted(DT))
    if op == "quantize":
        K = _between(rng, 16, 11008)
        return dict(op=op, M=_between(rng, 1, min(16384, 4097 * 11008 // K // (2 if x == "fp32" else 1))), K=K, x=x)
    if op in ("linear", "gemm"):
        N, K = _between(rng, 16, 11008), _between(rng, 16, 11008)
        M = _between(rng, 1, max(1, min(8192, 8192 * 11008 * 4096 // (N * K))))
        c = dict(op=op, M=M, N=N, K=K, x=x, y=y)
        if op == "gemm":
            del c["x"]
        return c
    k = rng.randint(1, 8)
    E = _between(rng, k, 128)
    if op == "experts":
        N, K = _between(rng, 64, 4096), _between(rng, 64, 4096)
        E = max(k, min(E, 8 * 4096 * 4096 // (N * K)))
        return dict(op=op, T=_between(rng, 1, max(1, 8192 // k)), k=k, E=E, N=N, K=K, y=y, drop=rng.choice([0.0, 0.1]))
    H = _between(rng, 64, 8192)
    most = 8191 * 4 * 4096 // (H * k) // (2 if x == "fp32" else 1)
    return dict(op=op, T=_between(rng, 1, max(1, min(16384, most))), k=k, E=E, H=H, x=x, drop=rng.choice([0.0, 0.1]))


def _pitch(K):
    """Bytes from one int8 row to the next: K rounded up to 64."""
    return -(-K // 64) * 64


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, M, K, dtype):
    """Normal values, every 128th channel ten times as large, one row in 32 all zeros (padding)."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, ::128] *= 10.0
    if M > 1:
        x[torch.rand(M, generator=g, device="cuda") < 1 / 32] = 0.0
    return x.to(dtype)


def _codes(g, rows, K, spread):
    """int8 rows at their pitch (the padding zero) and positive scales."""
    q = torch.zeros(rows, _pitch(K), dtype=torch.int8, device="cuda")
    q[:, :K] = (torch.randn(rows, K, generator=g, device="cuda") * 36).round().clamp(-127, 127).to(torch.int8)
    return q, (torch.rand(rows, generator=g, device="cuda") + 0.5) * spread


def _routing(g, T, k, E, drop):
    """int64 expert ids [T][k] as a top-k gives them, uneven over the experts, with dropped slots -1, and fp32 weights."""
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda") * 0.7
    top, ids = logits.topk(k, dim=1)
    weights = top.softmax(1)
    if drop:
        gone = torch.rand(T, k, generator=g, device="cuda") < drop / 2
        gone |= (torch.rand(T, generator=g, device="cuda") < drop / 2)[:, None]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids, weights


def _sorted_slots(ids, E):
    """(offsets [E+1], order [T*k], pos [T][k]), int32: slots sorted by expert, in slot order within one; dropped slots have pos -1
    and the order behind the last expert's rows is -1."""
    flat = ids.reshape(-1)
    n = flat.numel()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    at = torch.arange(n, device=flat.device)
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    pos = torch.empty_like(order)
    pos[order] = at
    pos = torch.where(kept, pos, torch.full_like(pos, -1))
    order = torch.where(at < offsets[E], order, torch.full_like(order, -1))
    return offsets.int(), order.int(), pos.int().view(ids.shape)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["xin"] = _activations(g, case["M"], case["K"], DT[case["x"]])
        return s
    if case["op"] in ("linear", "gemm"):
        if case["op"] == "linear":
            s["xin"] = _activations(g, case["M"], case["K"], DT[case["x"]])
        else:
            s["xq"], s["xs"] = _codes(g, case["M"], case["K"], 0.03)
        s["wq"], s["ws"] = _codes(g, case["N"], case["K"], 2e-4)
    else:
        ids, weights = _routing(g, case["T"], case["k"], case["E"], case["drop"])
        rows = case["T"] * case["k"]
        s["offsets"], s["order"], s["pos"] = _sorted_slots(ids, case["E"])
    if case["op"] == "experts":
        s["xq"], s["xs"] = _codes(g, case["T"], case["K"], 0.03)
        s["wq"], s["ws"] = _codes(g, case["E"] * case["N"], case["K"], 2e-4)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["out"] = torch.zeros(rows, case["N"], dtype=DT[case["y"]], device="cuda")
    elif case["op"] in ("route", "route_grad"):
        dt, H = DT[case["x"]], case["H"]
        s["weights"] = weights
        s["ys"] = torch.randn(rows, H, generator=g, device="cuda").to(dt)
        s["out"] = torch.zeros(rows, H, dtype=dt, device="cuda")
        if case["op"] == "route":
            s["ids"], s["xin"] = ids, _activations(g, case["T"], H, dt)
        else:
            s["dy"] = torch.randn(case["T"], H, generator=g, device="cuda").to(dt)
            s["dxs"] = torch.randn(rows, H, generator=g, device="cuda").to(dt)
    if own:
        import w4a16_gemv_amd as amd
        if "xq" in s:
            s["xt"] = amd.Int8Tensor(s["xq"], s["xs"], case["K"])
        if "wq" in s:
            s["wt"] = amd.Int8Tensor(s["wq"], s["ws"], case["K"])
        if case["op"] in ("experts", "route_grad"):
            s["plan"] = amd.MoeRoute(s["offsets"], s["order"], s["pos"])
    return s


def _quantized(x):
    """(codes as fp64, scale fp32): the products by the inverse in 64 bits, where they are exact next to a rounding border."""
    a = x.float().abs().amax(1).clamp_min(FLOOR)
    return (x.double() * (127.0 / a).double()[:, None]).round(), a / 127.0


def _scaled(acc, xs, ws, dtype):
    return (acc * xs.double()[..., None] * ws.double()[..., None, :]).to(dtype)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        q, scale = _quantized(s["xin"])
        return [(q.float() * scale[:, None]).to(s["xin"].dtype), scale]
    if op in ("linear", "gemm"):
        q, xs = _quantized(s["xin"]) if op == "linear" else (s["xq"][:, :s["K"]].double(), s["xs"])
        return [_scaled(q @ s["wq"][:, :s["K"]].double().t(), xs, s["ws"], DT[s["y"]])]
    if op == "experts":
        # each expert's rows at the head of a block of as many rows as the fullest expert has
        E, N, K, C = s["E"], s["N"], s["K"], max(1, s["most"])
        at = torch.arange(C, device="cuda")[None, :]
        row = (s["offsets"][:-1, None] + at).long()
        live = row < s["offsets"][1:, None]
        src = (s["order"][row.clamp(max=len(s["order"]) - 1)] // s["k"]).clamp_min(0).long()
        blocks = s["xq"][src][..., :K].double()
        acc = torch.bmm(blocks, s["wq"].view(E, N, -1)[..., :K].double().transpose(1, 2).contiguous())
        y = s["out"].clone()
        y[row[live]] = _scaled(acc, s["xs"][src], s["ws"].view(E, N), y.dtype)[live]
        return [y]
    k, out = s["k"], s["out"].clone()
    if op == "route":
        offsets, order, pos = _sorted_slots(s["ids"], s["E"])
        live = (order >= 0)[:, None]
        xs = torch.where(live, s["xin"][(order.long() // k).clamp_min(0)], out)
        w = torch.where(pos >= 0, s["weights"], torch.zeros_like(s["weights"]))
        y = (s["ys"][pos.long().clamp_min(0)].float() * w[..., None]).sum(1)
        return [offsets, order, pos, xs, y.to(out.dtype)]
    pos, kept = s["pos"].long(), s["pos"] >= 0
    at = pos.clamp_min(0)
    dy = s["dy"].float()
    out[pos[kept]] = (s["weights"][..., None] * dy[:, None, :])[kept].to(out.dtype)
    dw = torch.where(kept, (s["ys"][at].float() * dy[:, None, :]).sum(-1), torch.zeros_like(s["weights"]))
    dx = (s["dxs"][at].float() * kept[..., None].float()).sum(1)
    return [out, dw, dx.to(out.dtype)]


def run(state):
    if not own:
        return _plain(state)
    import w4a16_gemv_amd as amd
    s = state
    op = s["op"]
    if op == "quantize":
        t = amd.int8_quantize(s["xin"])
        return [t.dequant(out_dtype=DT[s["x"]]), t.scale]
    if op == "linear":
        return [amd.int8_linear(s["xin"], s["wt"], out_dtype=DT[s["y"]])]
    if op == "gemm":
        return [amd.int8_gemm(s["xt"], s["wt"], out_dtype=DT[s["y"]])]
    if op == "experts":
        return [amd.int8_gemm_grouped(s["xt"], s["wt"], s["plan"], y=s["out"])]
    if op == "route":
        plan = amd.moe_sort(s["ids"], s["E"])
        xs = amd.moe_gather(s["xin"], plan, out=s["out"])
        y = amd.moe_combine(s["ys"], plan, s["weights"])
        return [plan.offsets, plan.order, plan.pos, xs, y]
    dys, dw = amd.moe_combine_grad(s["dy"], s["ys"], s["plan"], s["weights"], dys=s["out"])
    return [dys, dw, amd.moe_gather_grad(s["dxs"], s["plan"])]


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": 2 * n * (SIZE[case["x"]] + 1) + 8 * case["M"], "flops": 4 * n}
    if op in ("linear", "gemm"):
        M, N, K = case["M"], case["N"], case["K"]
        x = M * K * SIZE[case["x"]] if op == "linear" else M * K + 4 * M
        return {"bytes": x + N * K + 4 * N + M * N * SIZE[case["y"]], "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    rows = int(T * k * (1 - case["drop"]))
    if op == "experts":
        N, K = case["N"], case["K"]
        # experts that T tokens reach, if each were as likely as another
        hit = E * (1 - (1 - k / E) ** T)
        return {"bytes": int(T * K + hit * N * K + rows * N * SIZE[case["y"]]), "flops": 2 * rows * N * K}
    H, b = case["H"], SIZE[case["x"]]
    if op == "route":
        return {"bytes": T * k * 20 + 4 * E + 2 * T * H * b + 2 * rows * H * b, "flops": 2 * rows * H}
    return {"bytes": T * k * 16 + 2 * T * H * b + 3 * rows * H * b, "flops": 4 * rows * H}


# --- the definitions in 64 bits ---------------------------------------------

def _codes_by_definition(x):
    """Codes (int64) and fp32 scales of a row, rounding by the remainder instead of by round()."""
    x = x.double()
    peak = torch.maximum(x.max(1).values, -x.min(1).values)
    peak = torch.where(peak < FLOOR, torch.full_like(peak, FLOOR), peak).float()
    scale, inverse = peak / 127, 127 / peak
    t = x * inverse.double().unsqueeze(1)
    low = torch.floor(t)
    rest = t - low
    up = (rest > 0.5) | ((rest == 0.5) & (low.long() % 2 != 0))
    return low.long() + up.long(), scale


def _whole_product(a, b):
    """a [M][K] times b [N][K] transposed, whole numbers up to 128, as fp64: pieces of 1024 columns are below 2^24 and so exact in fp32."""
    total = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for c in range(0, a.shape[1], 1024):
        total += (a[:, c:c + 1024].float() @ b[:, c:c + 1024].float().t()).double()
    return total


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, scale = _codes_by_definition(s["xin"])
        return [q.double() * scale.double().unsqueeze(1), scale.double()]
    if op in ("linear", "gemm"):
        if op == "linear":
            q, xs = _codes_by_definition(s["xin"])
        else:
            q, xs = s["xq"][:, :case["K"]], s["xs"]
        y = _whole_product(q, s["wq"][:, :case["K"]])
        y *= xs.double().unsqueeze(1)
        y *= s["ws"].double().unsqueeze(0)
        return [y]
    if op == "experts":
        N, K = case["N"], case["K"]
        y = torch.zeros(case["T"] * case["k"], N, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        token = s["order"].long() // case["k"]
        for e in range(case["E"]):
            a, b = ends[e], ends[e + 1]
            if a < b:
                t = token[a:b]
                w = s["wq"][e * N:(e + 1) * N, :K]
                y[a:b] = _whole_product(s["xq"][t, :K], w) * torch.outer(s["xs"][t].double(), s["ws"][e * N:(e + 1) * N].double())
        return [y]
    T, k, H = case["T"], case["k"], case["H"]
    if op == "route":
        slots = [(e, i) for i, e in enumerate(s["ids"].flatten().tolist()) if 0 <= e < case["E"]]
        slots.sort()
        counts = [0] * (case["E"] + 1)
        pos = [-1] * (T * k)
        for at, (e, i) in enumerate(slots):
            counts[e + 1] += 1
            pos[i] = at
        for e in range(case["E"]):
            counts[e + 1] += counts[e]
        order = [i for _, i in slots] + [-1] * (T * k - len(slots))
        whole = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (counts, order, pos)]
        xs = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        xs[:len(slots)] = s["xin"].double()[whole[1][:len(slots)].long() // k]
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        flat = whole[2].view(T, k).long()
        for j in range(k):
            on = flat[:, j] >= 0
            y[on] += s["weights"][on, j].double().unsqueeze(1) * s["ys"][flat[on, j]].double()
        return whole[:2] + [whole[2].view(T, k), xs, y]
    dys = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dy, flat = s["dy"].double(), s["pos"].long()
    for j in range(k):
        on = flat[:, j] >= 0
        at = flat[on, j]
        dys[at] = s["weights"][on, j].double().unsqueeze(1) * dy[on]
        dw[on, j] = torch.linalg.vecdot(s["ys"][at].double(), dy[on])
        dx[on] += s["dxs"][at].double()
    return [dys, dw, dx]
