"""The 8-bit integer products (include/int8.h): codes per token and per output
channel, int32 sums.

Argument marshalling only, as in _binding.py; work goes on torch's current
stream of the tensors' device, whichever device is current.  Nothing here is
recorded by autograd: tensors that require a gradient are refused while
gradients are being recorded, and so are those with a forward-mode tangent.
What a call writes (out, y, workspace) must not overlap its other tensors.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from ._binding import _check, _dev, _F32, load

_ROWS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I8 = (torch.int8,)


def _row_dtype(dtype: torch.dtype, name: str) -> int:
    code = _ROWS.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _on(dev: torch.device, t: torch.Tensor, name: str) -> None:
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _tangent(t: torch.Tensor) -> bool:
    """Whether t has a forward-mode tangent (which torch.no_grad() does not switch off)."""
    return (forward_ad._current_level >= 0 and torch._C._is_fwd_grad_enabled()
            and forward_ad.unpack_dual(t).tangent is not None)


def _no_grad(t: torch.Tensor, name: str) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which autograd would not see; call this under "
                         "torch.no_grad() or in a Function")
    if _tangent(t):
        raise ValueError(f"{name} has a forward-mode tangent, which the result would not; call this in a Function")


def _scale(t: "Int8Tensor", name: str) -> int:
    """The pointer of t's scales.  They were checked when t was made, but whether they
    require a gradient can change at any time."""
    s = t.scale
    if s.requires_grad or forward_ad._current_level >= 0:
        _no_grad(s, f"{name}.scale")
    return s.data_ptr()


def _gpu(t: torch.Tensor, name: str) -> int:
    """The pointer of a contiguous GPU tensor (of a type that was checked)."""
    if t.requires_grad or forward_ad._current_level >= 0:
        _no_grad(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _run(fn: str, dev: torch.device, *args) -> None:
    """One library call on the current stream of `dev`."""
    f = getattr(load(), fn)
    # the raw handle: torch.cuda.current_stream builds an object for it, which
    # costs as much as the rest of a small call's marshalling
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch._C._cuda_getDevice():
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st:
        _check(fn, st)


def _size(fn: str, dev: torch.device, *args) -> int:
    f = getattr(load(), fn)
    if dev.index == torch._C._cuda_getDevice():
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _scratch(workspace, fn: str, dev: torch.device, *sizes):
    """(pointer, bytes, tensor to keep until the call has returned) of the
    caller's workspace, or of one from torch's allocator."""
    if workspace is not None:
        _on(dev, workspace, "workspace")
        return _dev(workspace, "workspace", (torch.uint8,), 0), workspace.numel(), workspace
    nbytes = _size(fn, dev, *sizes)
    if nbytes == 0:
        return None, 0, None
    t = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return t.data_ptr(), nbytes, t


def int8_pitch(K: int) -> int:
    """Bytes from one row of codes to the next: K rounded up to 64."""
    return (int(K) + 63) // 64 * 64 if K > 0 else 0


class Int8Tensor:
    """Rows of int8 codes with one fp32 scale per row, on the GPU: a token's
    activations or an output channel's weights per row.

    data: int8 [rows][int8_pitch(K)], the bytes from K on zero; scale: fp32
    [rows]; value = code * scale.  int8_quantize makes one; codes from
    elsewhere (a checkpoint) are given here in that layout."""

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, K: int):
        K = int(K)
        if K < 0:
            raise ValueError(f"K must not be negative, got {K}")
        if data.dim() != 2 or data.shape[1] != int8_pitch(K):
            raise ValueError(f"data must be [rows, {int8_pitch(K)}] for K={K}, got shape "
                             f"{tuple(data.shape)}")
        rows = data.shape[0]
        _dev(data, "data", _I8, 0)
        _dev(scale, "scale", _F32, rows)
        if scale.numel() != rows:
            raise ValueError(f"scale has {scale.numel()} elements for {rows} rows")
        _on(data.device, scale, "scale")
        self.data, self.scale, self.K = data, scale, K

    @property
    def rows(self) -> int:
        return self.data.shape[0]

    @property
    def nbytes(self) -> int:
        return self.data.numel() + 4 * self.scale.numel()

    def dequant(self, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        return int8_dequant(self, out, out_dtype)

    def gemm(self, x, y=None, out_dtype: torch.dtype = torch.bfloat16, workspace=None):
        """The product of activations x with these weights: int8_gemm for an
        Int8Tensor, int8_linear for a tensor."""
        f = int8_gemm if isinstance(x, Int8Tensor) else int8_linear
        return f(x, self, y, out_dtype, workspace)


def int8_quantize(x: torch.Tensor, out: Int8Tensor | None = None) -> Int8Tensor:
    """Encode the rows of x (bf16, fp16 or fp32; the last dimension is K, the
    others are flattened) with one scale per row, on x's GPU.  out: an
    Int8Tensor of the same rows and K to write into."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    K = x.shape[-1]
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    code = _row_dtype(x.dtype, "x")
    if out is not None:
        _no_grad(out.scale, "out.scale")
    px, dev = _gpu(x, "x"), x.device
    if out is None:
        out = Int8Tensor.__new__(Int8Tensor)
        out.data = torch.empty((rows, int8_pitch(K)), dtype=torch.int8, device=dev)
        out.scale = torch.empty(rows, dtype=torch.float32, device=dev)
        out.K = K
    else:
        if out.rows != rows or out.K != K:
            raise ValueError(f"out is {out.rows} x {out.K}, expected {rows} x {K}")
        _on(dev, out.data, "out")
    _run("int8_quantize", dev, px, code, rows, K, out.data.data_ptr(), out.scale.data_ptr())
    return out


def int8_dequant(t: Int8Tensor, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of t's codes as [rows][K] in bf16, fp16 or fp32."""
    dev, rows, K, scale = t.data.device, t.data.shape[0], t.K, _scale(t, "t")
    if out is None:
        code = _row_dtype(out_dtype, "out_dtype")
        out = torch.empty((rows, K), dtype=out_dtype, device=dev)
    else:
        code = _row_dtype(out.dtype, "out")
        if out.shape != (rows, K):
            raise ValueError(f"out must be [{rows}, {K}], got shape {tuple(out.shape)}")
        _on(dev, out, "out")
    _run("int8_dequant", dev, t.data.data_ptr(), scale, rows, K, _gpu(out, "out"), code)
    return out


def _out(y, rows: int, N: int, dtype: torch.dtype, dev: torch.device):
    """(y, its pointer, its type code) with y allocated if it is None."""
    if y is None:
        code = _row_dtype(dtype, "out_dtype")
        y = torch.empty((rows, N), dtype=dtype, device=dev)
        return y, y.data_ptr(), code
    code = _row_dtype(y.dtype, "y")
    if y.shape != (rows, N):
        raise ValueError(f"y must be [{rows}, {N}], got shape {tuple(y.shape)}")
    _on(dev, y, "y")
    return y, _gpu(y, "y"), code


def int8_gemm_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for int8_gemm of an M x N x K product on `device` (None when
    the product would not use one).  Reusable by later calls of any shape on
    one stream (nothing is kept between calls); a shape that could use more
    splits its sums less, with the same bits."""
    return _workspace("int8_gemm_workspace_size", M, N, K, device)


def int8_linear_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for int8_linear of an M x N x K product on `device` (None
    when the product would not use one).  Reusable by later calls with no more
    rows and no larger K on one stream, as int8_gemm_workspace."""
    return _workspace("int8_linear_workspace_size", M, N, K, device)


def _workspace(fn, M, N, K, device):
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    nbytes = _size(fn, dev, int(M), int(N), int(K))
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def int8_gemm(x: Int8Tensor, w: Int8Tensor, y: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.bfloat16,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m][n] = (sum_k x[m][k] w[n][k]) * x.scale[m] * w.scale[n] for any
    number of rows of x; returns y [x.rows][w.rows] in out_dtype (or y's own).

    The integer sums are exact, so the bits do not depend on the workspace: a
    uint8 tensor from int8_gemm_workspace, or None for one from torch's
    allocator."""
    if x.K != w.K:
        raise ValueError(f"x has K={x.K}, w has K={w.K}")
    xs, ws = _scale(x, "x"), _scale(w, "w")
    xd, wd = x.data, w.data
    M, N, dev = xd.shape[0], wd.shape[0], xd.device
    _on(dev, wd, "w")
    y, py, code = _out(y, M, N, out_dtype, dev)
    pw, wbytes, _keep = _scratch(workspace, "int8_gemm_workspace_size", dev, M, N, x.K)
    _run("int8_gemm", dev, xd.data_ptr(), xs, wd.data_ptr(), ws, M, N, x.K, py, code, pw, wbytes)
    return y


def int8_linear(x: torch.Tensor, w: Int8Tensor, y: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """int8_gemm(int8_quantize(x), w) in one call, with the same bits: x is
    [M][K] (or [K], then y is [N]) in bf16, fp16 or fp32.

    workspace: a uint8 tensor from int8_linear_workspace, or None for one from
    torch's allocator."""
    one = x.dim() == 1
    if x.dim() > 2 or x.dim() < 1 or x.shape[-1] != w.K:
        raise ValueError(f"x must be [M, {w.K}] or [{w.K}], got shape {tuple(x.shape)}")
    xcode, ws = _row_dtype(x.dtype, "x"), _scale(w, "w")
    px, dev, wd = _gpu(x, "x"), x.device, w.data
    M, N = 1 if one else x.shape[0], wd.shape[0]
    _on(dev, wd, "w")
    flat = one and (y is None or y.dim() == 1)
    y2, py, code = _out(y.unsqueeze(0) if flat and y is not None else y, M, N, out_dtype, dev)
    pw, wbytes, _keep = _scratch(workspace, "int8_linear_workspace_size", dev, M, N, w.K)
    _run("int8_linear", dev, px, xcode, wd.data_ptr(), ws, M, N, w.K, py, code, pw, wbytes)
    if y is not None:
        return y
    return y2.view(N) if one else y2


def int8_gemm_grouped(x: Int8Tensor, w: Int8Tensor, route, y: torch.Tensor | None = None,
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
    xs, ws = _scale(x, "x"), _scale(w, "w")
    xd, wd, rows = x.data, w.data, route.rows
    N, dev = wd.shape[0] // E, xd.device
    _on(dev, wd, "w")
    _on(dev, route.offsets, "route")
    y, py, code = _out(y, rows, N, out_dtype, dev)
    _run("int8_gemm_grouped", dev, xd.data_ptr(), xs, xd.shape[0],
         None if x_sorted else route.order.data_ptr(), route.top_k, wd.data_ptr(),
         ws, route.offsets.data_ptr(), E, rows, N, x.K, py, code)
    return y
