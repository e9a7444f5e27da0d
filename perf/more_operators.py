"""The operators of 4-bit microscaled floats (E2M1 codes, one power of two to 32 of them) as measurable cases.

Each case is one pass through one operator, in two forms: the plain form in elementary torch operations (`own`
false) and the calls a user makes of w4a16_gemv_amd (`own` true).  `exact` computes the same outputs in 64 bits
from the definitions.

The format: a code is a sign and one of the magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6; the codes of a row come in blocks of
32 with one byte E as their scale, value = code * 2^(E - 127).  Two codes lie in a byte, the earlier one in its low half.

Operators (the case's "op"):
  quantize  rows to codes and scales, and back to the values that they stand for: E - 127 = floor(log2(max|x|)) - 2 of
            a block (-127 at least), code = x * 2^(127 - E) rounded to the nearest magnitude, ties to the even code, past
            6 to 6.
  linear    activations quantized on the way into the product with weights in this format.
  gemm      the same product from activations that are quantized already.
  gemv      the product of activations as they are with weights in this format.
  experts   the product of quantized activations for rows sorted by expert, each expert with weights of its own; the
            activations are read in token order through the routing's order.
  mlp       an expert layer for a few tokens: y[t] = sum_j weights[t][j] * W2[e] act(W1[e] x[t]) with e = ids[t][j]; act
            is silu(g) * u of the first and second half of W1's channels (gated), or silu.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step's token ahead of a projection
        dict(name="quantize_token", op="quantize", M=1, K=4096, x="bf16"),
        # the inner activation of an MLP over a long prompt, an odd number of rows
        dict(name="quantize_prompt", op="quantize", M=4097, K=11008, x="bf16"),
        # single-token decode of an attention projection with 4-bit activations
        dict(name="linear_token", op="linear", M=1, N=4096, K=4096, x="bf16", y="bf16"),
        # sizes that no tile and no block divides, everything in fp32
        dict(name="linear_ragged", op="linear", M=333, N=4099, K=1501, x="fp32", y="fp32"),
        # a long prompt through an MLP projection, quantized once for gate and up
        dict(name="gemm_prompt", op="gemm", M=8192, N=11008, K=4096, y="bf16"),
        # single-token decode of an MLP projection, only the weights in 4 bits
        dict(name="gemv_token", op="gemv", M=1, N=11008, K=4096, x="bf16", y="bf16"),
        # seven sequences through the MLP's way down
        dict(name="gemv_batch", op="gemv", M=7, N=4096, K=11008, x="fp16", y="fp16"),
        # a decode step of 16 sequences over many small experts: few rows each, most experts' weights read
        dict(name="experts_step", op="experts", T=16, k=4, E=64, N=1024, K=2048, y="bf16", drop=0.0),
        # a prompt over a few large experts with uneven loads
        dict(name="experts_prompt", op="experts", T=4096, k=2, E=8, N=4096, K=4096, y="bf16", drop=0.0),
        # single-token decode through two of eight large experts
        dict(name="mlp_token", op="mlp", T=1, k=2, E=8, H=4096, F=11008, gated=True, x="bf16", drop=0.0),
        # three sequences over small experts of odd widths without a gate, some slots of other ranks' experts
        dict(name="mlp_ragged", op="mlp", T=3, k=4, E=64, H=1001, F=333, gated=False, x="fp32", drop=0.2),
        # a decode step of 16 sequences over many small experts
        dict(name="mlp_step", op="mlp", T=16, k=4, E=64, H=2048, F=1024, gated=True, x="bf16", drop=0.0),
    ]


def _between(rng, lo, hi):
    """A whole number, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "gemm", "gemv", "experts", "mlp"])
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
    if op == "gemv":
        return dict(op=op, M=rng.randint(1, 16), N=_between(rng, 16, 11008), K=_between(rng, 16, 11008), x=x, y=y)
    k = rng.randint(1, 8)
    E = _between(rng, k, 128)
    drop = rng.choice([0.0, 0.1])
    if op == "experts":
        N, K = _between(rng, 64, 4096), _between(rng, 64, 4096)
        E = max(k, min(E, 8 * 4096 * 4096 // (N * K)))
        return dict(op=op, T=_between(rng, 1, max(1, 8192 // k)), k=k, E=E, N=N, K=K, y=y, drop=drop)
    H, F = _between(rng, 64, 4096), _between(rng, 64, 11008)
    E = max(k, min(E, 8 * 4096 * 11008 // (H * F)))
    # the slots' weights are what a pass costs: no more than those of 16 tokens with four experts of 2048 x 1024 each
    T = _between(rng, 1, max(1, min(64, 64 * 2048 * 1024 // (H * F * k))))
    return dict(op=op, T=T, k=k, E=E, H=H, F=F, gated=rng.random() < 0.7, x=x, drop=drop)


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


def _encode(x):
    """(codes uint8 [rows][blocks][16], scales uint8 [rows][blocks]) of fp32 rows; a last block that is short is filled up with zeros."""
    rows, K = x.shape
    blocks = -(-K // BLOCK)
    if blocks * BLOCK != K:
        x = torch.cat([x, torch.zeros(rows, blocks * BLOCK - K, dtype=x.dtype, device=x.device)], 1)
    x = x.view(rows, blocks, BLOCK)
    a = x.abs()
    e = ((a.amax(2).view(torch.int32) >> 23) - 2).clamp_min(0)
    a = torch.ldexp(a, (127 - e)[..., None])
    # half way between two magnitudes goes to the even code: up from 0.75, 1.75 and 3.5, down from the others
    code = (a > 0.25).byte()
    for border, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if up else (a > border)
    code |= (x.view(torch.int32) < 0).byte() << 3
    return code[..., 0::2] | code[..., 1::2] << 4, e.byte()


def _weights(g, rows, K, spread):
    """Normal values in the format, in pieces of at most 2^27 values."""
    blocks = -(-K // BLOCK)
    codes = torch.empty(rows, blocks, BLOCK // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, blocks, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // K)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        codes[a:b], scales[a:b] = _encode(torch.randn(b - a, K, generator=g, device="cuda") * spread)
    return codes, scales


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
    op = case["op"]
    if op == "quantize":
        s["xin"] = _activations(g, case["M"], case["K"], DT[case["x"]])
    elif op in ("linear", "gemm", "gemv"):
        if op == "gemm":
            s["xc"] = _encode(_activations(g, case["M"], case["K"], torch.float32))
        else:
            s["xin"] = _activations(g, case["M"], case["K"], DT[case["x"]])
        s["wc"] = _weights(g, case["N"], case["K"], 0.02)
    else:
        ids, weights = _routing(g, case["T"], case["k"], case["E"], case["drop"])
        if op == "experts":
            s["offsets"], s["order"], s["pos"] = _sorted_slots(ids, case["E"])
            s["xc"] = _encode(_activations(g, case["T"], case["K"], torch.float32))
            s["wc"] = _weights(g, case["E"] * case["N"], case["K"], 0.02)
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
            s["out"] = torch.zeros(case["T"] * case["k"], case["N"], dtype=DT[case["y"]], device="cuda")
        else:
            s["ids"], s["weights"] = ids, weights
            s["xin"] = _activations(g, case["T"], case["H"], DT[case["x"]])
            s["w1c"] = _weights(g, case["E"] * case["F"] * (2 if case["gated"] else 1), case["H"], 0.02)
            s["w2c"] = _weights(g, case["E"] * case["H"], case["F"], 0.02)
    if own:
        import w4a16_gemv_amd as amd
        for name, K in (("xc", "K"), ("wc", "K"), ("w1c", "H"), ("w2c", "F")):
            if name in s:
                s[name[:-1]] = amd.Mxfp4Tensor.from_blocks(*s[name], case[K])
        if op == "experts":
            s["plan"] = amd.MoeRoute(s["offsets"], s["order"], s["pos"])
    return s


def _table(device, dtype):
    return torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=dtype, device=device)


def _values(codes, scales, K):
    """fp32 [rows][K] of codes [rows][blocks][16]."""
    v = _table(codes.device, torch.float32)[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(2)
    v = torch.ldexp(v, (scales.int() - 127)[..., None]).flatten(1)
    return v[:, :K]


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return [_values(*_encode(s["xin"].float()), s["K"]).to(s["xin"].dtype)]
    if op in ("linear", "gemm", "gemv"):
        K = s["K"]
        x = s["xin"].float() if op == "gemv" else _values(*(s["xc"] if op == "gemm" else _encode(s["xin"].float())), K)
        return [(x @ _values(*s["wc"], K).t()).to(DT[s["y"]])]
    if op == "experts":
        # each expert's rows at the head of a block of as many rows as the fullest expert has
        E, N, K, C = s["E"], s["N"], s["K"], max(1, s["most"])
        at = torch.arange(C, device="cuda")[None, :]
        row = (s["offsets"][:-1, None] + at).long()
        live = row < s["offsets"][1:, None]
        src = (s["order"][row.clamp(max=len(s["order"]) - 1)] // s["k"]).clamp_min(0).long()
        w = _values(*s["wc"], K).reshape(E, N, K).transpose(1, 2).contiguous()
        acc = torch.bmm(_values(*s["xc"], K)[src], w)
        y = s["out"].clone()
        y[row[live]] = acc[live].to(y.dtype)
        return [y]
    T, k, E, H, F = s["T"], s["k"], s["E"], s["H"], s["F"]
    ids = s["ids"].reshape(-1)
    kept = (ids >= 0) & (ids < E)
    at = torch.where(kept, ids, torch.zeros_like(ids))

    def slots(w, rows, K):  # each slot's expert's weights [T * k][rows][K]
        codes, scales = (t.view(E, rows, *t.shape[1:])[at] for t in w)
        return _values(codes.flatten(0, 1), scales.flatten(0, 1), K).reshape(T * k, rows, K)

    x = s["xin"].float().repeat_interleave(k, 0)
    h = torch.bmm(slots(s["w1c"], F * (2 if s["gated"] else 1), H), x[:, :, None])[..., 0]
    h = _silu(h[:, :F]) * h[:, F:] if s["gated"] else _silu(h)
    o = torch.bmm(slots(s["w2c"], H, F), h[:, :, None])[..., 0]
    w = torch.where(kept, s["weights"].reshape(-1), torch.zeros_like(s["weights"].reshape(-1)))
    return [(o * w[:, None]).view(T, k, H).sum(1).to(s["xin"].dtype)]


def run(state):
    if not own:
        return _plain(state)
    import w4a16_gemv_amd as amd
    s = state
    op = s["op"]
    if op == "quantize":
        return [amd.mxfp4_quantize(s["xin"]).dequant(out_dtype=DT[s["x"]])]
    if op == "linear":
        return [amd.mxfp4_linear(s["xin"], s["w"], out_dtype=DT[s["y"]])]
    if op == "gemm":
        return [amd.mxfp4_gemm(s["x"], s["w"], out_dtype=DT[s["y"]])]
    if op == "gemv":
        return [amd.mxfp4_gemv(s["xin"], s["w"], out_dtype=DT[s["y"]])]
    if op == "experts":
        return [amd.mxfp4_gemm_grouped(s["x"], s["w"], s["plan"], y=s["out"])]
    return [amd.mxfp4_moe_mlp(s["xin"], s["w1"], s["w2"], s["ids"], s["weights"])]


def _bytes(rows, K):
    return rows * -(-K // BLOCK) * (BLOCK // 2 + 1)


def work(case):
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": 2 * (M * K * SIZE[case["x"]] + _bytes(M, K)), "flops": 4 * M * K}
    if op in ("linear", "gemm", "gemv"):
        M, N, K = case["M"], case["N"], case["K"]
        x = _bytes(M, K) if op == "gemm" else M * K * SIZE[case["x"]]
        return {"bytes": x + _bytes(N, K) + M * N * SIZE[case["y"]], "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    rows = max(1, int(T * k * (1 - case["drop"])))
    # experts that T tokens reach, if each were as likely as another
    hit = E * (1 - (1 - k / E) ** T)
    if op == "experts":
        N, K = case["N"], case["K"]
        return {"bytes": int(_bytes(T, K) + hit * _bytes(N, K) + rows * N * SIZE[case["y"]]), "flops": 2 * rows * N * K}
    H, F, up = case["H"], case["F"], 2 if case["gated"] else 1
    return {"bytes": int(hit * (_bytes(up * F, H) + _bytes(H, F)) + 2 * T * H * SIZE[case["x"]] + 12 * T * k),
            "flops": 2 * rows * (up + 1) * H * F}


# --- the definitions in 64 bits ---------------------------------------------

def _definition(x):
    """What rows stand for after encoding, fp64: each value next to the nearest multiple of its interval's step."""
    rows, K = x.shape
    full = torch.zeros(rows, -(-K // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:, :K] = x.double()
    v = full.view(rows, -1, BLOCK)
    peak = torch.maximum(v.max(2).values, -v.min(2).values)
    power = torch.where(peak > 0, torch.frexp(peak).exponent - 3, torch.full_like(peak, -127, dtype=torch.int32))
    unit = torch.pow(2.0, power.clamp_min(-127).double()).unsqueeze(2)
    t = (v / unit).abs()
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0)).double()
    low = torch.floor(t / step)
    rest = t / step - low
    up = (rest > 0.5) | ((rest == 0.5) & (low.long() % 2 != 0))
    near = torch.where(t >= 6, torch.full_like(t, 6.0), (low + up.double()) * step)
    return (torch.sign(v) * near * unit).view(rows, -1)[:, :K]


def _stand_for(w, K, first=0, count=None):
    """fp64 [count][K] of the rows from `first` on."""
    codes, scales = (t[first:first + (t.shape[0] if count is None else count)] for t in w)
    out = torch.empty(*scales.shape, BLOCK, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        m, e = (c & 1).double(), (c >> 1 & 3).double()
        size = torch.where(e > 0, torch.pow(2.0, e - 1) * (1 + m / 2), m / 2)
        out[..., half::2] = torch.where(c >= 8, -size, size)
    out *= torch.pow(2.0, scales.double() - 127).unsqueeze(2)
    return out.view(scales.shape[0], -1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return [_definition(s["xin"])]
    if op in ("linear", "gemm", "gemv"):
        K = case["K"]
        x = _definition(s["xin"]) if op == "linear" else _stand_for(s["xc"], K) if op == "gemm" else s["xin"].double()
        return [torch.nn.functional.linear(x, _stand_for(s["wc"], K))]
    if op == "experts":
        N, K = case["N"], case["K"]
        y = torch.zeros(case["T"] * case["k"], N, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        x, token = _stand_for(s["xc"], K), s["order"].long() // case["k"]
        for e in range(case["E"]):
            a, b = ends[e], ends[e + 1]
            if a < b:
                y[a:b] = torch.nn.functional.linear(x[token[a:b]], _stand_for(s["wc"], K, e * N, N))
        return [y]
    H, F, up = case["H"], case["F"], 2 if case["gated"] else 1
    y = torch.zeros(case["T"], H, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        at, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if len(at):
            v = torch.nn.functional.linear(s["xin"][at].double(), _stand_for(s["w1c"], H, e * up * F, up * F))
            g = v[:, :F]
            h = g * torch.sigmoid(g)
            if case["gated"]:
                h = h * v[:, F:]
            o = torch.nn.functional.linear(h, _stand_for(s["w2c"], F, e * H, H))
            y.index_add_(0, at, o * s["weights"][at, slot].double().unsqueeze(1))
    return [y]
