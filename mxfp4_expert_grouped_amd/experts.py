"""Experts in 16 bits with gradients (moe_linear_rows and its two gradients).

    y = linear(x, w, offsets)        # row r times the matrix of its expert

Every call goes to the current stream of its tensors' GPU; nothing is
synchronised, so all of it can be captured into a graph.  What :mod:`.tokens`
says of a backward pass that is captured holds here too: capture the forward
pass with it on leaves of its own, or call the ``_backward`` functions, which
use no autograd.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import mxmoe as M
from .layer import ROW_DTYPES, device_index, in_memory, on_device

_PRODUCT_DTYPES = (torch.bfloat16, torch.float16)

_workspace_bytes = lru_cache(maxsize=1024)(M.moe_linear_rows_workspace_bytes)


def _rows(x: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """A matrix with dense rows that do not overlap, on 16 bytes (else a copy), and its row stride"""
    x = in_memory(x)
    rows, cols = x.shape
    ld, step = x.stride()
    if rows == 0 or cols == 0:
        return x, cols
    if (step != 1 and cols > 1) or (ld < cols and rows > 1) or ld > 1 << 21 or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
        ld = cols
    return x, ld if rows > 1 else cols


def _dense(w: torch.Tensor) -> torch.Tensor:
    w = in_memory(w).contiguous()
    return w.clone() if w.data_ptr() % 16 and w.numel() else w


def _check_product(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor], cols: int, what: str) -> Tuple[int, int, int]:
    """-> (matrices, n, k) of w, for x [R, cols] with cols = ``what`` of w"""
    if x.dtype not in _PRODUCT_DTYPES:
        raise ValueError(f"expected bfloat16 or float16 rows, got {x.dtype}")
    if w.dtype != x.dtype:
        raise ValueError(f"rows are {x.dtype}, weights {w.dtype}")
    if w.dim() != (2 if offsets is None else 3):
        raise ValueError(f"weights must be [N, K] without offsets and [E, N, K] with them, got {list(w.shape)}")
    mats, (n, k) = (1 if offsets is None else w.shape[0]), w.shape[-2:]
    if x.dim() != 2 or x.shape[1] != (k if what == "K" else n):
        raise ValueError(f"expected rows [R, {k if what == 'K' else n}], got {list(x.shape)}")
    _check_offsets(offsets, mats)
    return mats, n, k


def _check_offsets(offsets: Optional[torch.Tensor], mats: int) -> None:
    if offsets is not None and (offsets.dtype is not torch.int32 or offsets.shape != (mats + 1,)):
        raise ValueError(f"offsets must be int32 [{mats + 1}], got {offsets.dtype} {list(offsets.shape)}")


def _workspace(device: torch.device, *shape: int) -> Tuple[Optional[torch.Tensor], int]:
    need = _workspace_bytes(*shape)
    return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need


def _linear(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor], back: bool) -> torch.Tensor:
    """x W^T, or dy W where ``back``"""
    mats, n, k = _check_product(x, w, offsets, x.shape[-1], "N" if back else "K")
    dev = device_index(x, w, offsets)
    x, ld = _rows(x)
    w = _dense(w)
    if offsets is not None:
        offsets = offsets.contiguous()
    rows, cols = x.shape[0], (k if back else n)
    out = torch.empty(rows, cols, dtype=x.dtype, device=x.device)
    dt = ROW_DTYPES[x.dtype]
    ws, need = _workspace(x.device, M.MOE_ROWS_INPUT if back else M.MOE_ROWS_FORWARD, dt, rows, ld, 0, mats,
                          offsets is not None, n, k, dt, cols)
    on_device(dev, M.moe_linear_rows_dx if back else M.moe_linear_rows, x.data_ptr(), dt, rows, ld, w.data_ptr(), mats,
              None if offsets is None else offsets.data_ptr(), n, k, out.data_ptr(), cols,
              None if ws is None else ws.data_ptr(), need)
    return out


def linear_dx(dy: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of :func:`linear` in the rows: dx [R, K] from dy [R, N]; rows of no expert are zero."""
    return _linear(dy, w, offsets, True)


def linear_dw(dy: torch.Tensor, x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
              dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Gradient of :func:`linear` in the weights: dw [E, N, K] (without offsets [N, K]) from dy [R, N] and
    x [R, K], of dy's type or float32 (``dtype``); an expert without rows has a zero gradient."""
    if dy.dtype not in _PRODUCT_DTYPES or x.dtype != dy.dtype:
        raise ValueError(f"expected bfloat16 or float16 gradients and rows of the same type, got {dy.dtype} and {x.dtype}")
    dtype = dtype or dy.dtype
    if dtype not in (dy.dtype, torch.float32):
        raise ValueError(f"the gradient of the weights is {dy.dtype} or float32, not {dtype}")
    if dy.dim() != 2 or x.dim() != 2 or x.shape[0] != dy.shape[0]:
        raise ValueError(f"expected gradients [R, N] and rows [R, K], got {list(dy.shape)} and {list(x.shape)}")
    if offsets is not None and (offsets.dim() != 1 or offsets.numel() < 2):
        raise ValueError(f"offsets must be int32 [E + 1], got {list(offsets.shape)}")
    mats = 1 if offsets is None else offsets.numel() - 1
    _check_offsets(offsets, mats)
    dev = device_index(dy, x, offsets)
    dy, ld_dy = _rows(dy)
    x, ld_x = _rows(x)
    if offsets is not None:
        offsets = offsets.contiguous()
    (rows, n), k = dy.shape, x.shape[1]
    out = torch.empty((n, k) if offsets is None else (mats, n, k), dtype=dtype, device=dy.device)
    dt, out_dt = ROW_DTYPES[dy.dtype], ROW_DTYPES[dtype]
    ws, need = _workspace(dy.device, M.MOE_ROWS_WEIGHT, dt, rows, ld_dy, ld_x, mats, offsets is not None, n, k, out_dt, k)
    on_device(dev, M.moe_linear_rows_dw, dy.data_ptr(), dt, rows, ld_dy, x.data_ptr(), ld_x, mats,
              None if offsets is None else offsets.data_ptr(), n, k, out.data_ptr(), out_dt,
              None if ws is None else ws.data_ptr(), need)
    return out


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        need_x, need_w = x.requires_grad, w.requires_grad
        ctx.save_for_backward(x if need_w else None, w if need_x else None, offsets)
        return _linear(x, w, offsets, False)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dx = linear_dx(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = linear_dw(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def linear(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor] = None, checkpoint=None) -> torch.Tensor:
    """Rows times the matrix of their expert, y [R, N] of x's type (bfloat16 or float16), sums in fp32.

    x [R, K]; w [N, K], or [E, N, K] with ``offsets`` int32 [E+1]: rows offsets[e] .. offsets[e+1]-1 take
    matrix e (:func:`.tokens.sort_tokens`); rows of no expert give zeros.  Differentiable in x and w.
    """
    if not (torch.is_grad_enabled() and (x.requires_grad or w.requires_grad)):
        return _linear(x, w, offsets, False)
    return _Linear.apply(x, w, offsets)
