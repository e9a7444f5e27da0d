"""The 8-bit integer products (include/int8.h): codes per token and per output
channel, int32 sums.

Argument marshalling only, as in _binding.py; work goes on torch's current
stream of the tensors' device, whichever device is current.  Nothing here is
recorded by autograd.
"""
from __future__ import annotations

import torch

from ._binding import _check, _dev, _F32, load

_ROWS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I8 = (torch.int8,)


def _row_dtype(dtype: torch.dtype, name: str) -> int:
    code = _ROWS.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _same_device(dev: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _run(fn: str, dev: torch.device, *args) -> None:
    """One library call on the current stream of `dev`."""
    f = getattr(load(), fn)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if dev.index == torch.cuda.current_device():
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st:
        _check(fn, st)


def _size(fn: str, dev: torch.device, *args) -> int:
    f = getattr(load(), fn)
    if dev.index == torch.cuda.current_device():
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _scratch(workspace, nbytes: int, dev: torch.device):
    """(pointer, bytes, tensor to keep until the call has returned) of the
    caller's workspace, or of one from torch's allocator."""
    if workspace is not None:
        _same_device(dev, workspace=workspace)
        return _dev(workspace, "workspace", (torch.uint8,), 0), workspace.numel(), workspace
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
        _same_device(data.device, scale=scale)
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
    px = _dev(x, "x", (x.dtype,), rows * K)
    dev = x.device
    if out is None:
        out = Int8Tensor.__new__(Int8Tensor)
        out.data = torch.empty((rows, int8_pitch(K)), dtype=torch.int8, device=dev)
        out.scale = torch.empty(rows, dtype=torch.float32, device=dev)
        out.K = K
    elif out.rows != rows or out.K != K:
        raise ValueError(f"out is {out.rows} x {out.K}, expected {rows} x {K}")
    _same_device(dev, out=out.data)
    _run("int8_quantize", dev, px, code, rows, K, out.data.data_ptr(), out.scale.data_ptr())
    return out


def int8_dequant(t: Int8Tensor, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of t's codes as [rows][K] in bf16, fp16 or fp32."""
    dev = t.data.device
    if out is None:
        out = torch.empty((t.rows, t.K), dtype=out_dtype, device=dev)
    code = _row_dtype(out.dtype, "out")
    if tuple(out.shape) != (t.rows, t.K):
        raise ValueError(f"out must be [{t.rows}, {t.K}], got shape {tuple(out.shape)}")
    _same_device(dev, out=out)
    _run("int8_dequant", dev, t.data.data_ptr(), t.scale.data_ptr(), t.rows, t.K,
         _dev(out, "out", (out.dtype,), 0), code)
    return out


def _out(y, rows: int, N: int, dtype: torch.dtype, dev: torch.device):
    """(y, its type code) with y allocated if it is None."""
    if y is None:
        code = _row_dtype(dtype, "out_dtype")
        return torch.empty((rows, N), dtype=dtype, device=dev), code
    code = _row_dtype(y.dtype, "y")
    if tuple(y.shape) != (rows, N):
        raise ValueError(f"y must be [{rows}, {N}], got shape {tuple(y.shape)}")
    _same_device(dev, y=y)
    _dev(y, "y", (y.dtype,), 0)
    return y, code


def int8_gemm_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for int8_gemm of an M x N x K product on `device` (None when
    the product would not use one).  Reusable by later calls of the same or
    smaller shapes on one stream (nothing is kept between calls)."""
    return _workspace("int8_gemm_workspace_size", M, N, K, device)


def int8_linear_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for int8_linear, as int8_gemm_workspace."""
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
    M, N, dev = x.rows, w.rows, x.data.device
    _same_device(dev, w=w.data)
    y, code = _out(y, M, N, out_dtype, dev)
    pw, wbytes, _keep = _scratch(workspace, _size("int8_gemm_workspace_size", dev, M, N, x.K)
                                 if workspace is None else 0, dev)
    _run("int8_gemm", dev, x.data.data_ptr(), x.scale.data_ptr(), w.data.data_ptr(),
         w.scale.data_ptr(), M, N, x.K, y.data_ptr(), code, pw, wbytes)
    return y


def int8_linear(x: torch.Tensor, w: Int8Tensor, y: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """int8_gemm(int8_quantize(x), w) in one call, with the same bits: x is
    [M][K] (or [K], then y is [N]) in bf16, fp16 or fp32.

    workspace: a uint8 tensor from int8_linear_workspace, or None for one from
    torch's allocator."""
    if x.dim() not in (1, 2) or x.shape[-1] != w.K:
        raise ValueError(f"x must be [M, {w.K}] or [{w.K}], got shape {tuple(x.shape)}")
    M, N, dev = 1 if x.dim() == 1 else x.shape[0], w.rows, x.device
    xcode = _row_dtype(x.dtype, "x")
    px = _dev(x, "x", (x.dtype,), 0)
    _same_device(dev, w=w.data)
    if y is not None and x.dim() == 1 and y.dim() == 1:
        _out(y.unsqueeze(0), M, N, out_dtype, dev)
        y2, code = y, _ROWS[y.dtype]
    else:
        y2, code = _out(y, M, N, out_dtype, dev)
    pw, wbytes, _keep = _scratch(workspace, _size("int8_linear_workspace_size", dev, M, N, w.K)
                                 if workspace is None else 0, dev)
    _run("int8_linear", dev, px, xcode, w.data.data_ptr(), w.scale.data_ptr(), M, N, w.K,
         y2.data_ptr(), code, pw, wbytes)
    return y2.view(N) if x.dim() == 1 and y is None else y2


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
    N, dev = w.rows // E, x.data.device
    _same_device(dev, w=w.data, route=route.offsets)
    y, code = _out(y, route.rows, N, out_dtype, dev)
    _run("int8_gemm_grouped", dev, x.data.data_ptr(), x.scale.data_ptr(), x.rows,
         None if x_sorted else route.order.data_ptr(), route.top_k, w.data.data_ptr(),
         w.scale.data_ptr(), route.offsets.data_ptr(), E, route.rows, N, x.K, y.data_ptr(), code)
    return y
