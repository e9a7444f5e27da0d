"""Routing around expert products (include/moe.h): slots sorted by expert, rows
moved into that order and back with the router's weights, and the gradients.

Argument marshalling only, as in _binding.py; work goes on torch's current
stream of the tensors' device, whichever device is current.  Nothing here is
recorded by autograd: a program that trains calls moe_combine_grad and
moe_gather_grad in its backward pass, and tensors that require a gradient are
refused while gradients are being recorded.  Those with a forward-mode tangent
are refused too.  What a call writes (out, dys, workspace) must not overlap its
other tensors.
"""
from __future__ import annotations

import torch

from ._binding import _dev
from ._int8 import _gpu, _on, _row_dtype, _run, _scratch

_I32 = (torch.int32,)
_IDS = {torch.int32: 4, torch.int64: 8}


class MoeRoute:
    """Where the slots of a batch went (moe_sort): T tokens with top_k slots
    each, over `experts` experts.

    offsets: int32 [experts + 1], expert e has the sorted rows [offsets[e],
    offsets[e + 1]); order: int32 [T * top_k], the flat slot t * top_k + j of
    each sorted row, -1 behind the last expert's; pos: int32 [T][top_k], the
    sorted row of each slot, -1 for a dropped one."""

    def __init__(self, offsets: torch.Tensor, order: torch.Tensor, pos: torch.Tensor):
        if pos.dim() != 2 or pos.shape[1] < 1:
            raise ValueError(f"pos must be [T, top_k], got shape {tuple(pos.shape)}")
        _dev(pos, "pos", _I32, 0)
        _dev(order, "order", _I32, 0)
        _dev(offsets, "offsets", _I32, 1)
        if order.numel() != pos.numel():
            raise ValueError(f"order has {order.numel()} elements, pos {pos.numel()}")
        _on(pos.device, offsets, "offsets")
        _on(pos.device, order, "order")
        self.offsets, self.order, self.pos = offsets, order, pos

    @property
    def T(self) -> int:
        return self.pos.shape[0]

    @property
    def top_k(self) -> int:
        return self.pos.shape[1]

    @property
    def rows(self) -> int:
        """Rows of a buffer in sorted order: one for each slot, dropped or not."""
        return self.order.numel()

    @property
    def experts(self) -> int:
        return self.offsets.numel() - 1


def moe_sort(ids: torch.Tensor, experts: int, workspace: torch.Tensor | None = None) -> MoeRoute:
    """Sort the slots of ids (int32 or int64 [T][top_k]) by expert, stable.
    Ids outside [0, experts) are dropped slots.  workspace: a uint8 tensor of
    moe_sort_workspace_size bytes, or None for one from torch's allocator."""
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError(f"ids must be [T, top_k], got shape {tuple(ids.shape)}")
    T, top_k = ids.shape
    experts = int(experts)
    if experts < 0:
        raise ValueError(f"experts must not be negative, got {experts}")
    if ids.dtype not in _IDS:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    pi, dev = _gpu(ids, "ids"), ids.device
    route = MoeRoute.__new__(MoeRoute)
    route.offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    route.order = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    route.pos = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    pw, nbytes, _keep = _scratch(workspace, "moe_sort_workspace_size", dev, T, top_k, experts)
    _run("moe_sort", dev, pi, _IDS[ids.dtype], T, top_k, experts, route.offsets.data_ptr(),
         route.order.data_ptr(), route.pos.data_ptr(), pw, nbytes)
    return route


def _no_grad(fn: str, *tensors) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{fn}: a tensor requires a gradient, which autograd would not see; call it under "
                         "torch.no_grad() or in a Function, and its gradient function in the backward pass")


def _rows(t: torch.Tensor, name: str, rows: int, H: int, dev, dtype) -> int:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, H):
        raise ValueError(f"{name} must be [{rows}, {H}], got shape {tuple(t.shape)}")
    _on(dev, t, name)
    return _gpu(t, name)


def moe_gather(x: torch.Tensor, route: MoeRoute, out: torch.Tensor | None = None) -> torch.Tensor:
    """x's rows ([T][H]: bf16, fp16 or fp32) in sorted order, [route.rows][H];
    rows that no slot has are left as they were (undefined where out is None)."""
    _no_grad("moe_gather", x, out)
    if x.dim() != 2:
        raise ValueError(f"x must be [T, H], got shape {tuple(x.shape)}")
    dev, dtype, H, pos = x.device, x.dtype, x.shape[1], route.pos
    (T, k), code = pos.shape, _row_dtype(x.dtype, "x")
    px = _rows(x, "x", T, H, dev, dtype)
    _on(dev, pos, "route")
    if out is None:
        out = torch.empty((T * k, H), dtype=dtype, device=dev)
    po = _rows(out, "out", T * k, H, dev, dtype)
    _run("moe_gather", dev, px, code, pos.data_ptr(), T, k, T * k, H, po)
    return out


def moe_combine(ys: torch.Tensor, route: MoeRoute, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j weights[t][j] ys[pos[t][j]] ([T][H]) over the slots of each
    token that have a row; weights: fp32 [T][top_k], or None for ones."""
    _no_grad("moe_combine", ys, weights, out)
    if ys.dim() != 2:
        raise ValueError(f"ys must be [rows, H], got shape {tuple(ys.shape)}")
    dev, dtype, H, pos = ys.device, ys.dtype, ys.shape[1], route.pos
    (T, k), code = pos.shape, _row_dtype(ys.dtype, "ys")
    ps = _rows(ys, "ys", T * k, H, dev, dtype)
    _on(dev, pos, "route")
    pw = None if weights is None else _rows(weights, "weights", T, k, dev, torch.float32)
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=dev)
    po = _rows(out, "out", T, H, dev, dtype)
    _run("moe_combine", dev, ps, code, pw, pos.data_ptr(), T, k, T * k, H, po)
    return out


def moe_gather_grad(dxs: torch.Tensor, route: MoeRoute,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of moe_gather: dx[t] = sum_j dxs[pos[t][j]]."""
    return moe_combine(dxs, route, None, out)


def moe_combine_grad(dy: torch.Tensor, ys: torch.Tensor, route: MoeRoute,
                     weights: torch.Tensor | None = None, dys: torch.Tensor | None = None):
    """The gradients (dys [route.rows][H], dweights fp32 [T][top_k]) of
    moe_combine, given dy [T][H] and its inputs.  Rows of dys that no slot has
    are left as they were (undefined where dys is None)."""
    _no_grad("moe_combine_grad", dy, ys, weights, dys)
    if dy.dim() != 2:
        raise ValueError(f"dy must be [T, H], got shape {tuple(dy.shape)}")
    dev, dtype, H, pos = dy.device, dy.dtype, dy.shape[1], route.pos
    (T, k), code = pos.shape, _row_dtype(dy.dtype, "dy")
    pg = _rows(dy, "dy", T, H, dev, dtype)
    ps = _rows(ys, "ys", T * k, H, dev, dtype)
    _on(dev, pos, "route")
    pw = None if weights is None else _rows(weights, "weights", T, k, dev, torch.float32)
    if dys is None:
        dys = torch.empty((T * k, H), dtype=dtype, device=dev)
    po = _rows(dys, "dys", T * k, H, dev, dtype)
    dweights = torch.empty((T, k), dtype=torch.float32, device=dev)
    _run("moe_combine_grad", dev, pg, ps, code, pw, pos.data_ptr(), T, k, T * k, H, po, dweights.data_ptr())
    return dys, dweights
