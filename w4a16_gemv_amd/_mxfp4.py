"""The 4-bit microscaled floats (include/mxfp4.h): E2M1 codes with a power of two
to every 32 of a row, their products, and the expert layer of a few tokens.

Argument marshalling only, as in _binding.py; work goes on torch's current
stream of the tensors' device, whichever device is current.  Nothing here is
recorded by autograd: tensors that require a gradient are refused while
gradients are being recorded, and so are those with a forward-mode tangent.
What a call writes (out, y, workspace) must not overlap its other tensors.
"""
from __future__ import annotations

import torch

from ._binding import _U8, _dev
from ._int8 import _gpu, _on, _out, _row_dtype, _run, _scratch, _workspace
from ._moe import _IDS

_BLOCK = 32


def mxfp4_pitch(K: int) -> int:
    """Bytes from one row of codes to the next: K rounded up to 128, halved."""
    return (int(K) + 127) // 128 * 64 if K > 0 else 0


def mxfp4_scale_size(rows: int, K: int) -> int:
    """Bytes of the scales of rows of K elements: 256 to every 32 rows x 256 elements."""
    return (int(rows) + 31) // 32 * ((int(K) + 255) // 256) * 256 if rows > 0 and K > 0 else 0


def _tiled(scales: torch.Tensor) -> torch.Tensor:
    """Scales [rows][blocks] in the order of Mxfp4Tensor.scale."""
    rows, blocks = scales.shape
    tiles, steps = -(-rows // 32), -(-blocks // 8)
    full = torch.zeros((tiles * 32, steps * 8), dtype=torch.uint8, device=scales.device)
    full[:rows, :blocks] = scales
    # [tile][row][step][half][byte] to [tile][step][half][row][byte]
    return full.view(tiles, 32, steps, 2, 4).permute(0, 2, 3, 1, 4).contiguous().view(-1)


class Mxfp4Tensor:
    """Rows of 4-bit codes with one power of two to every 32 of them, on the GPU: a
    token's activations or an output channel's weights per row.

    data: uint8 [rows][mxfp4_pitch(K)], two codes to a byte, the earlier one in its
    low half, those from K on zero; scale: uint8 [mxfp4_scale_size(rows, K)], the
    exponents (biased by 127; 255 for NaN) in tiles as include/mxfp4.h lays them
    out.  mxfp4_quantize makes one; from_blocks takes codes and scales of a
    checkpoint in their usual order."""

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, K: int):
        K = int(K)
        if K < 0:
            raise ValueError(f"K must not be negative, got {K}")
        if data.dim() != 2 or data.shape[1] != mxfp4_pitch(K):
            raise ValueError(f"data must be [rows, {mxfp4_pitch(K)}] for K={K}, got shape {tuple(data.shape)}")
        size = mxfp4_scale_size(data.shape[0], K)
        if scale.dim() != 1 or scale.numel() != size:
            raise ValueError(f"scale must be [{size}] for {data.shape[0]} rows of K={K}, got shape {tuple(scale.shape)}")
        _dev(data, "data", _U8, 0)
        _dev(scale, "scale", _U8, 0)
        _on(data.device, scale, "scale")
        self.data, self.scale, self.K = data, scale, K

    @classmethod
    def _empty(cls, rows: int, K: int, dev: torch.device) -> "Mxfp4Tensor":
        t = cls.__new__(cls)
        t.data = torch.empty((rows, mxfp4_pitch(K)), dtype=torch.uint8, device=dev)
        t.scale = torch.empty(mxfp4_scale_size(rows, K), dtype=torch.uint8, device=dev)
        t.K = K
        return t

    @classmethod
    def from_blocks(cls, codes: torch.Tensor, scales: torch.Tensor, K: int | None = None) -> "Mxfp4Tensor":
        """From codes uint8 [rows][blocks][16] (two to a byte, the earlier one in its
        low half) and scales uint8 [rows][blocks], laid out once.  K: the elements
        of a row where the last block is not full (its codes from K on count as
        zero); None for all of them."""
        if codes.dim() != 3 or codes.shape[2] != _BLOCK // 2:
            raise ValueError(f"codes must be [rows, blocks, 16], got shape {tuple(codes.shape)}")
        rows, blocks = codes.shape[:2]
        if scales.shape != (rows, blocks):
            raise ValueError(f"scales must be [{rows}, {blocks}], got shape {tuple(scales.shape)}")
        K = blocks * _BLOCK if K is None else int(K)
        if K < 0 or -(-K // _BLOCK) != blocks:
            raise ValueError(f"rows of K={K} have {-(-K // _BLOCK)} blocks, got {blocks}")
        for t, name in ((codes, "codes"), (scales, "scales")):
            if t.dtype != torch.uint8:
                raise ValueError(f"{name} must be uint8, got {t.dtype}")
            if not t.is_cuda:
                raise ValueError(f"{name} must be on the GPU, got {t.device}")
        _on(codes.device, scales, "scales")
        with torch.cuda.device(codes.device):
            data = torch.zeros((rows, mxfp4_pitch(K)), dtype=torch.uint8, device=codes.device)
            n = blocks * _BLOCK // 2
            data[:, :n] = codes.reshape(rows, n)
            if K % _BLOCK:
                data[:, (K + 1) // 2:] = 0
                if K % 2:
                    data[:, K // 2] &= 15
            return cls(data, _tiled(scales), K)

    def blocks(self) -> tuple[torch.Tensor, torch.Tensor]:
        """(codes uint8 [rows][blocks][16], scales uint8 [rows][blocks]) in their usual order."""
        rows, blocks = self.rows, -(-self.K // _BLOCK)
        tiles, steps = -(-rows // 32), -(-self.K // 256)
        codes = self.data[:, :blocks * _BLOCK // 2].reshape(rows, blocks, _BLOCK // 2)
        scales = self.scale.view(tiles, steps, 2, 32, 4).permute(0, 3, 1, 2, 4).reshape(tiles * 32, steps * 8)
        return codes.contiguous(), scales[:rows, :blocks].contiguous()

    @property
    def rows(self) -> int:
        return self.data.shape[0]

    @property
    def nbytes(self) -> int:
        return self.data.numel() + self.scale.numel()

    def dequant(self, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        return mxfp4_dequant(self, out, out_dtype)

    def gemm(self, x, y=None, out_dtype: torch.dtype = torch.bfloat16, workspace=None):
        """The product of activations x with these weights: mxfp4_gemm for an
        Mxfp4Tensor, mxfp4_linear for a tensor."""
        f = mxfp4_gemm if isinstance(x, Mxfp4Tensor) else mxfp4_linear
        return f(x, self, y, out_dtype, workspace)

    def gemv(self, x, y=None, out_dtype: torch.dtype = torch.bfloat16):
        """The product of up to 16 rows of activations as they are with these weights."""
        return mxfp4_gemv(x, self, y, out_dtype)


def mxfp4_quantize(x: torch.Tensor, out: Mxfp4Tensor | None = None) -> Mxfp4Tensor:
    """Encode the rows of x (bf16, fp16 or fp32; the last dimension is K, the
    others are flattened) in blocks of 32, on x's GPU.  out: an Mxfp4Tensor of
    the same rows and K to write into."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    K = x.shape[-1]
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    code = _row_dtype(x.dtype, "x")
    px, dev = _gpu(x, "x"), x.device
    if out is None:
        out = Mxfp4Tensor._empty(rows, K, dev)
    else:
        if out.rows != rows or out.K != K:
            raise ValueError(f"out is {out.rows} x {out.K}, expected {rows} x {K}")
        _on(dev, out.data, "out")
    _run("mxfp4_quantize", dev, px, code, rows, K, out.data.data_ptr(), out.scale.data_ptr())
    return out


def mxfp4_dequant(t: Mxfp4Tensor, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of t's codes as [rows][K] in bf16, fp16 or fp32."""
    dev, rows, K = t.data.device, t.data.shape[0], t.K
    if out is None:
        code = _row_dtype(out_dtype, "out_dtype")
        out = torch.empty((rows, K), dtype=out_dtype, device=dev)
    else:
        code = _row_dtype(out.dtype, "out")
        if out.shape != (rows, K):
            raise ValueError(f"out must be [{rows}, {K}], got shape {tuple(out.shape)}")
        _on(dev, out, "out")
    _run("mxfp4_dequant", dev, t.data.data_ptr(), t.scale.data_ptr(), rows, K, _gpu(out, "out"), code)
    return out


def mxfp4_gemm_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for mxfp4_gemm of an M x N x K product on `device` (None when
    the product would not use one).  Reusable by later calls of any shape on
    one stream (nothing is kept between calls); a shape that could use more
    splits its sums less, which may change their last bits."""
    return _workspace("mxfp4_gemm_workspace_size", M, N, K, device)


def mxfp4_linear_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for mxfp4_linear of an M x N x K product on `device` (None
    when the product would not use one; few rows of few channels do not).  Reusable
    by later calls with no more rows and no larger K on one stream, as
    mxfp4_gemm_workspace."""
    return _workspace("mxfp4_linear_workspace_size", M, N, K, device)


def mxfp4_gemm(x: Mxfp4Tensor, w: Mxfp4Tensor, y: torch.Tensor | None = None,
               out_dtype: torch.dtype = torch.bfloat16,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m][n] = sum_k x[m][k] w[n][k] of the values of both for any number of
    rows of x, summed in fp32; returns y [x.rows][w.rows] in out_dtype (or y's
    own).  workspace: a uint8 tensor from mxfp4_gemm_workspace, or None for one
    from torch's allocator."""
    if x.K != w.K:
        raise ValueError(f"x has K={x.K}, w has K={w.K}")
    xd, wd = x.data, w.data
    M, N, dev = xd.shape[0], wd.shape[0], xd.device
    _on(dev, wd, "w")
    y, py, code = _out(y, M, N, out_dtype, dev)
    pw, wbytes, _keep = _scratch(workspace, "mxfp4_gemm_workspace_size", dev, M, N, x.K)
    _run("mxfp4_gemm", dev, xd.data_ptr(), x.scale.data_ptr(), wd.data_ptr(), w.scale.data_ptr(), M, N, x.K, py, code,
         pw, wbytes)
    return y


def _vectors(x: torch.Tensor, w: Mxfp4Tensor, y, out_dtype):
    """(x's pointer and type code, rows, whether x is a vector, y as [M][N], y's pointer and type code)."""
    one = x.dim() == 1
    if x.dim() > 2 or x.dim() < 1 or x.shape[-1] != w.K:
        raise ValueError(f"x must be [M, {w.K}] or [{w.K}], got shape {tuple(x.shape)}")
    xcode = _row_dtype(x.dtype, "x")
    px, dev, wd = _gpu(x, "x"), x.device, w.data
    M, N = 1 if one else x.shape[0], wd.shape[0]
    _on(dev, wd, "w")
    flat = one and y is not None and y.dim() == 1
    y2, py, code = _out(y.unsqueeze(0) if flat else y, M, N, out_dtype, dev)
    return px, xcode, M, one, y2, py, code


def mxfp4_linear(x: torch.Tensor, w: Mxfp4Tensor, y: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """mxfp4_gemm(mxfp4_quantize(x), w) in one call: x is [M][K] (or [K], then y
    is [N]) in bf16, fp16 or fp32.  The codes are the same; the order of the fp32
    sums may be another.

    workspace: a uint8 tensor from mxfp4_linear_workspace, or None for one from
    torch's allocator."""
    px, xcode, M, one, y2, py, code = _vectors(x, w, y, out_dtype)
    dev, N = x.device, w.data.shape[0]
    pw, wbytes, _keep = _scratch(workspace, "mxfp4_linear_workspace_size", dev, M, N, w.K)
    _run("mxfp4_linear", dev, px, xcode, w.data.data_ptr(), w.scale.data_ptr(), M, N, w.K, py, code, pw, wbytes)
    if y is not None:
        return y
    return y2.view(N) if one else y2


def mxfp4_gemv(x: torch.Tensor, w: Mxfp4Tensor, y: torch.Tensor | None = None,
               out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y[m][n] = sum_k x[m][k] w[n][k] with the activations as they are, for up to
    16 rows: x is [M][K] (or [K], then y is [N]) in bf16, fp16 or fp32.  The
    products are exact, the sums fp32."""
    px, xcode, M, one, y2, py, code = _vectors(x, w, y, out_dtype)
    if M > 16:
        raise ValueError(f"x has {M} rows, at most 16 are taken; mxfp4_linear takes any number")
    N = w.data.shape[0]
    _run("mxfp4_gemv", x.device, px, xcode, w.data.data_ptr(), w.scale.data_ptr(), M, N, w.K, py, code)
    if y is not None:
        return y
    return y2.view(N) if one else y2


def mxfp4_gemm_grouped(x: Mxfp4Tensor, w: Mxfp4Tensor, route, y: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.bfloat16,
                       x_sorted: bool = False) -> torch.Tensor:
    """The product where each sorted row has its expert's weights: row i of y,
    of expert e, is x's row of the token of sorted row i times w's rows
    [e N, (e + 1) N).

    x: the tokens' rows (route.T of them), read where they lie; with x_sorted
    one row per sorted row instead (route.rows of them).  w: the experts' rows
    one after the other (route.experts * N rows).  route: from moe_sort.
    Returns y [route.rows][N]; rows that no expert has (dropped slots leave
    them at the end) are left as they were, undefined where y is None."""
    E = route.experts
    if E == 0 or w.rows % E:
        raise ValueError(f"w has {w.rows} rows, not a multiple of {E} experts")
    if x.K != w.K:
        raise ValueError(f"x has K={x.K}, w has K={w.K}")
    want = route.rows if x_sorted else route.T
    if x.rows != want:
        raise ValueError(f"x has {x.rows} rows, expected {want}")
    xd, wd, rows = x.data, w.data, route.rows
    N, dev = wd.shape[0] // E, xd.device
    _on(dev, wd, "w")
    _on(dev, route.offsets, "route")
    y, py, code = _out(y, rows, N, out_dtype, dev)
    _run("mxfp4_gemm_grouped", dev, xd.data_ptr(), x.scale.data_ptr(), xd.shape[0],
         None if x_sorted else route.order.data_ptr(), route.top_k, wd.data_ptr(), w.scale.data_ptr(),
         route.offsets.data_ptr(), E, rows, N, x.K, py, code)
    return y


def mxfp4_moe_mlp(x: torch.Tensor, w1: Mxfp4Tensor, w2: Mxfp4Tensor, ids: torch.Tensor,
                  weights: torch.Tensor | None = None, y: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The expert layer of up to 64 tokens in two launches, activations as they are:
    y[t] = sum_j weights[t][j] W2[e] act(W1[e] x[t]) with e = ids[t][j].

    x: [T][H] in bf16, fp16 or fp32.  w2: the experts' rows one after the other, H
    of each (E * H rows of F).  w1: E * F rows of H, act is silu; or E * 2 F, of each
    expert the gate's rows first, act is silu(gate) * other.  ids: int32 or int64
    [T][top_k] with top_k <= 32; ids outside [0, E) are dropped slots.  weights: fp32
    [T][top_k], or None for ones.  Returns y [T][H] in x's type.  workspace: a uint8
    tensor of mxfp4_moe_mlp_workspace_size bytes, or None for one from torch's
    allocator.  Past about 16 tokens mxfp4_gemm_grouped of quantized activations takes
    less time."""
    if x.dim() != 2:
        raise ValueError(f"x must be [T, H], got shape {tuple(x.shape)}")
    T, H = x.shape
    code = _row_dtype(x.dtype, "x")
    px, dev = _gpu(x, "x"), x.device
    F = w2.K
    if w1.K != H:
        raise ValueError(f"w1 has K={w1.K}, x has {H} values to a row")
    if H == 0 or w2.rows % H:
        raise ValueError(f"w2 has {w2.rows} rows, not a multiple of {H}")
    E = w2.rows // H
    if w1.rows not in (E * F, 2 * E * F):
        raise ValueError(f"w1 has {w1.rows} rows, expected {E * F} or, with a gate, {2 * E * F}")
    if ids.dim() != 2 or ids.shape[0] != T or ids.shape[1] < 1:
        raise ValueError(f"ids must be [{T}, top_k], got shape {tuple(ids.shape)}")
    if ids.dtype not in _IDS:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    top_k = ids.shape[1]
    if T > 64 or top_k > 32:
        raise ValueError(f"at most 64 tokens with 32 slots each are taken, got {T} with {top_k}; "
                         "mxfp4_gemm_grouped takes any number")
    for t, name in ((w1.data, "w1"), (w2.data, "w2"), (ids, "ids")):
        _on(dev, t, name)
    pw = None
    if weights is not None:
        if weights.dtype != torch.float32 or weights.shape != ids.shape:
            raise ValueError(f"weights must be float32 {list(ids.shape)}, got {weights.dtype} {list(weights.shape)}")
        _on(dev, weights, "weights")
        pw = _gpu(weights, "weights")
    if y is not None and y.dtype != x.dtype:
        raise ValueError(f"y must be {x.dtype}, got {y.dtype}")
    y, py, _ = _out(y, T, H, x.dtype, dev)
    ps, nbytes, _keep = _scratch(workspace, "mxfp4_moe_mlp_workspace_size", dev, T, top_k, E, H, F, code)
    _run("mxfp4_moe_mlp", dev, px, code, w1.data.data_ptr(), w1.scale.data_ptr(), w2.data.data_ptr(),
         w2.scale.data_ptr(), _gpu(ids, "ids"), _IDS[ids.dtype], pw, T, top_k, E, H, F, int(w1.rows != E * F), py, ps,
         nbytes)
    return y
