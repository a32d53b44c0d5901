"""Tokens sorted by expert and back, with gradients (moe_sort_tokens,
moe_dispatch_rows, moe_combine_rows and moe_combine_rows_backward).

    order = sort_tokens(ids, num_experts)          # ids [T, k] from a router
    xs = dispatch(x, order)                        # [T*k, d], sorted by expert
    rows = ...                                     # expert e has rows offsets[e] .. offsets[e+1]-1
    y = combine(rows, weights, order)              # [T, d]

``dispatch`` and ``combine`` are differentiable (x; rows and weights), once and
backwards: tensors with a forward-mode tangent are refused.
Every call goes to the current stream of its tensors' GPU; nothing is
synchronised, so all of it can be captured into a graph.  A backward pass that
is captured needs leaves that no graph built outside the capture still holds
(autograd would bring that graph's stream into the capture): capture the
forward pass with it on ``x.detach().requires_grad_()``, or call
``dispatch_backward`` and ``combine_backward``, which use no autograd.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import mxmoe as M
from .layer import device_index, in_memory, on_device, row_dtype


class TokenOrder:
    """Which row belongs to which (token, choice): see moe_sort_tokens.  Fixed once
    it is made; the calls go by its tensors' addresses, so these are checked here."""
    __slots__ = ("offsets", "row_src", "token_row")

    def __init__(self, offsets: torch.Tensor, row_src: torch.Tensor, token_row: torch.Tensor):
        for name, t, dims in (("offsets", offsets, 1), ("row_src", row_src, 1), ("token_row", token_row, 2)):
            if t.dtype is not torch.int32 or t.dim() != dims or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of {dims} dimensions")
            if t.device != token_row.device:
                raise ValueError(f"tensors on different devices: {t.device} and {token_row.device}")
        if offsets.numel() < 2 or row_src.numel() != token_row.numel():
            raise ValueError(f"offsets {list(offsets.shape)}, row_src {list(row_src.shape)} and token_row "
                             f"{list(token_row.shape)} are not [E+1], [T*k] and [T, k]")
        _set_offsets(self, offsets)      # int32 [E+1] first row of each expert; offsets[E] rows in all
        _set_row_src(self, row_src)      # int32 [T*k] pair t*k + j of each row, -1 behind the last
        _set_token_row(self, token_row)  # int32 [T, k] row of each pair, -1 for a dropped one

    def __setattr__(self, name, value):
        raise AttributeError("a TokenOrder does not change: make another one")

    def __reduce__(self):
        return TokenOrder, (self.offsets, self.row_src, self.token_row)

    @property
    def num_experts(self) -> int:
        return self.offsets.numel() - 1

    @property
    def num_tokens(self) -> int:
        return self.token_row.shape[0]

    @property
    def top_k(self) -> int:
        return self.token_row.shape[1]

    @property
    def capacity(self) -> int:
        """Rows of a buffer that holds every pair."""
        return self.token_row.numel()

    def _num_rows(self) -> int:
        return self.offsets.data_ptr() + 4 * self.num_experts


# (the slots' own setters: __setattr__ refuses)
_set_offsets, _set_row_src, _set_token_row = (TokenOrder.__dict__[n].__set__ for n in TokenOrder.__slots__)


_new = TokenOrder.__new__


def _own_order(offsets: torch.Tensor, row_src: torch.Tensor, token_row: torch.Tensor) -> TokenOrder:
    """An order of tensors made here (the checks take a tenth of a small call)."""
    order = _new(TokenOrder)
    _set_offsets(order, offsets)
    _set_row_src(order, row_src)
    _set_token_row(order, token_row)
    return order


_sort_workspace = lru_cache(maxsize=256)(M.moe_sort_tokens_workspace_bytes)


def sort_tokens(ids: torch.Tensor, num_experts: int) -> TokenOrder:
    """The order of the pairs of ``ids`` (int32 or int64 [T, k]) sorted by expert;
    ids outside [0, num_experts) are dropped (-1: padding)."""
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"ids must be int32 or int64 [T, k], got {ids.dtype} with {ids.dim()} dimensions")
    dev = device_index(ids)
    if not ids.is_contiguous():
        ids = ids.contiguous()
    t, k = ids.shape
    need = _sort_workspace(t, k, num_experts)
    device = ids.device
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=device)
    row_src = torch.empty(t * k, dtype=torch.int32, device=device)
    token_row = torch.empty(t, k, dtype=torch.int32, device=device)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    on_device(dev, M.moe_sort_tokens, ids.data_ptr(),
              M.MOE_ID_INT64 if ids.dtype is torch.int64 else M.MOE_ID_INT32, t, k, num_experts, offsets.data_ptr(),
              row_src.data_ptr(), token_row.data_ptr(), ws.data_ptr() if need else None, need)
    return _own_order(offsets, row_src, token_row)


def _matrix(x: torch.Tensor, rows: int, what: str):
    """x [rows, d] with dense rows that do not overlap (else a copy), and its row stride"""
    if x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"{what} must be [{rows}, d], got {tuple(x.shape)}")
    d = x.shape[1]
    x = in_memory(x)
    ld, step = x.stride()
    if d == 0 or rows == 0:
        return x, d
    if step == 1 and (ld >= d or rows == 1):
        return x, max(ld, d)
    return x.contiguous(), d


def _dispatch(x: torch.Tensor, order: TokenOrder) -> torch.Tensor:
    dev = device_index(x, order.token_row)
    tr = order.token_row
    t, k = tr.shape
    x, ld = _matrix(x, t, "x")
    d = x.shape[1]
    xs = torch.empty(t * k, d, dtype=x.dtype, device=x.device)
    sz = x.element_size()
    on_device(dev, M.moe_dispatch_rows, x.data_ptr(), d * sz, ld * sz, tr.data_ptr(), t, k, order._num_rows(), t * k,
              xs.data_ptr(), d * sz)
    return xs


def _combine(rows: torch.Tensor, weights: Optional[torch.Tensor], order: TokenOrder) -> torch.Tensor:
    dev = device_index(rows, weights, order.token_row)
    tr = order.token_row
    t, k = tr.shape
    rows, ld = _matrix(rows, t * k, "rows")
    if weights is not None:
        weights = (weights.resolve_neg() if weights.is_neg() else weights).contiguous()
    d = rows.shape[1]
    y = torch.empty(t, d, dtype=rows.dtype, device=rows.device)
    on_device(dev, M.moe_combine_rows, rows.data_ptr(), row_dtype(rows.dtype), t * k, d, ld, tr.data_ptr(),
              weights.data_ptr() if weights is not None else None, t, k, y.data_ptr(), d)
    return y


def dispatch_backward(dxs: torch.Tensor, order: TokenOrder) -> torch.Tensor:
    """Gradient of :func:`dispatch`: dx [T, d] from dxs [T*k, d]."""
    return _combine(dxs, None, order)


def combine_backward(dy: torch.Tensor, rows: Optional[torch.Tensor], weights: Optional[torch.Tensor],
                     order: TokenOrder, need_rows: bool = True, need_weights: bool = True):
    """Gradients of :func:`combine` from dy [T, d]: (drows [T*k, d] or None, dweights [T, k] or None).
    ``rows`` is needed for dweights only."""
    t, k = order.token_row.shape
    dt = row_dtype(dy.dtype)
    if need_weights:
        if rows is None or rows.dtype != dy.dtype or rows.dim() != 2 or rows.shape[1] != dy.shape[-1]:
            raise ValueError("the gradient of the weights needs rows of dy's type and width")
    else:
        rows = None
    _check_weights(weights, order)
    dev = device_index(dy, rows, weights, order.token_row)
    dy, ld_dy = _matrix(dy, t, "dy")
    d = ld_rows = dy.shape[1]
    if rows is not None:
        rows, ld_rows = _matrix(rows, t * k, "rows")
    if weights is not None:
        weights = (weights.resolve_neg() if weights.is_neg() else weights).contiguous()
    drows = torch.empty(t * k, d, dtype=dy.dtype, device=dy.device) if need_rows else None
    dw = torch.empty(t, k, dtype=torch.float32, device=dy.device) if need_weights else None
    ptr = lambda x: x.data_ptr() if x is not None else None  # noqa: E731
    on_device(dev, M.moe_combine_rows_backward, dy.data_ptr(), ptr(rows), dt, t * k, d, ld_dy, ld_rows,
              order.token_row.data_ptr(), ptr(weights), t, k, order._num_rows(), ptr(drows), d, ptr(dw))
    return drows, dw


def _check_weights(weights: Optional[torch.Tensor], order: TokenOrder) -> None:
    if weights is not None and (weights.dtype is not torch.float32 or weights.shape != order.token_row.shape):
        raise ValueError(f"weights must be float32 {list(order.token_row.shape)}, got {weights.dtype} {list(weights.shape)}")


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        # saved as tensors, so that a change of the order in place before the backward pass is an error
        ctx.save_for_backward(order.offsets, order.row_src, order.token_row)
        return _dispatch(x, order)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        return _combine(dxs, None, _own_order(*ctx.saved_tensors)), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, order):
        need_w = weights is not None and weights.requires_grad
        ctx.save_for_backward(rows if need_w else None, weights, order.offsets, order.row_src, order.token_row)
        return _combine(rows, weights, order)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, weights, *order = ctx.saved_tensors
        need_rows, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        return (*combine_backward(dy, rows, weights, _own_order(*order), need_rows, need_w), None)


def dispatch(x: torch.Tensor, order: TokenOrder) -> torch.Tensor:
    """xs [T*k, d]: row r is the row of x of the token that ``order.row_src[r]`` belongs to; zeros behind
    the last row.  Any element type moves (MXFP4 codes and scales too); bf16, fp16 and fp32 have a gradient,
    dx[t] = sum of its rows' gradients in fp32."""
    if not (x.requires_grad and torch.is_grad_enabled()):
        return _dispatch(x, order)
    row_dtype(x.dtype)
    return _Dispatch.apply(x, order)


def combine(rows: torch.Tensor, weights: Optional[torch.Tensor], order: TokenOrder) -> torch.Tensor:
    """y [T, d]: the sum of a token's rows [T*k, d] (bf16, fp16 or fp32) times their float32 weights [T, k]
    (None: ones), in fp32, rounded once; a token whose pairs are all dropped gets zeros."""
    row_dtype(rows.dtype)
    _check_weights(weights, order)
    if not (torch.is_grad_enabled() and (rows.requires_grad or (weights is not None and weights.requires_grad))):
        return _combine(rows, weights, order)
    return _Combine.apply(rows, weights, order)
