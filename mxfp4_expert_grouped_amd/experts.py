"""Experts in 16 bits with gradients (moe_linear_rows, moe_swiglu and their
gradients), and activations kept in 8 bits for them (moe_quantize_mx8).

    order = tokens.sort_tokens(ids, num_experts)
    xs = tokens.dispatch(x, order)                   # rows sorted by expert
    h = linear(xs, w_gate_up, order.offsets)         # row r times the matrix of its expert
    o = linear(swiglu(h), w_down, order.offsets)
    y = tokens.combine(o, weights, order)

``checkpoint="mx8"`` keeps what the backward pass needs of the rows in MXFP8,
about half the bytes of their own type: E4M3 elements with one E8M0 scale per
32 columns, whose values then stand for the rows in the gradients.  ``mlp`` is
the three lines in the middle with nothing else kept.

Every call goes to the current stream of its tensors' GPU; nothing is
synchronised, so all of it can be captured into a graph.  What :mod:`.tokens`
says of a backward pass that is captured holds here too: capture the forward
pass with it on leaves of its own, or call the ``_backward`` functions, which
use no autograd.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple, Union

import torch
from torch.autograd.function import once_differentiable

from . import mxmoe as M
from .layer import ROW_DTYPES, device_index, in_memory, on_device, row_dtype

# codes [R, C] and scales [R, S], uint8
Kept = Tuple[torch.Tensor, torch.Tensor]

_PRODUCT_DTYPES = (torch.bfloat16, torch.float16)

_forward_bytes = lru_cache(maxsize=1024)(M.moe_linear_rows_workspace_bytes)
_backward_bytes = lru_cache(maxsize=1024)(M.moe_linear_rows_backward_workspace_bytes)


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


def _strided(x: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """A matrix with dense rows that do not overlap (else a copy), and its row stride"""
    x = in_memory(x)
    rows, cols = x.shape
    ld, step = x.stride()
    if rows == 0 or cols == 0:
        return x, cols
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        return x.contiguous(), cols
    return x, ld if rows > 1 else cols


def _dense(w: torch.Tensor) -> torch.Tensor:
    w = in_memory(w).contiguous()
    return w.clone() if w.data_ptr() % 16 and w.numel() else w


def _check_weights(w: torch.Tensor, offsets: Optional[torch.Tensor], dtype: torch.dtype) -> Tuple[int, int, int]:
    """-> (matrices, n, k) of w, for rows of type dtype"""
    if dtype not in _PRODUCT_DTYPES:
        raise ValueError(f"expected bfloat16 or float16 rows, got {dtype}")
    if w.dtype != dtype:
        raise ValueError(f"rows are {dtype}, weights {w.dtype}")
    if w.dim() != (2 if offsets is None else 3):
        raise ValueError(f"weights must be [N, K] without offsets and [E, N, K] with them, got {list(w.shape)}")
    return (1, *w.shape) if offsets is None else tuple(w.shape)


def _check_offsets(offsets: Optional[torch.Tensor], mats: int) -> Optional[torch.Tensor]:
    if offsets is None:
        return None
    if offsets.dtype is not torch.int32 or offsets.shape != (mats + 1,):
        raise ValueError(f"offsets must be int32 [{mats + 1}], got {offsets.dtype} {list(offsets.shape)}")
    return offsets.contiguous()


def _scratch(need: int, like: torch.Tensor) -> Optional[torch.Tensor]:
    return torch.empty(need, dtype=torch.uint8, device=like.device) if need else None


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _linear(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor]) -> torch.Tensor:
    mats, n, k = _check_weights(w, offsets, x.dtype)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"expected rows [R, {k}], got {list(x.shape)}")
    offsets = _check_offsets(offsets, mats)
    dev = device_index(x, w, offsets)
    x, ld = _rows(x)
    w = _dense(w)
    rows, dt = x.shape[0], ROW_DTYPES[x.dtype]
    y = torch.empty(rows, n, dtype=x.dtype, device=x.device)
    need = _forward_bytes(dt, rows, ld, mats, offsets is not None, n, k, n)
    ws = _scratch(need, x)
    on_device(dev, M.moe_linear_rows, x.data_ptr(), dt, rows, ld, w.data_ptr(), mats, _ptr(offsets), n, k, y.data_ptr(), n,
              _ptr(ws), need)
    return y


def _is_kept(x) -> bool:
    return isinstance(x, (tuple, list))


def _kept(x: Kept, cols: Optional[int] = None, scales: int = 0) -> Kept:
    """Contiguous codes [R, cols] and scales [R, scales], without cols those of any matrix"""
    if len(x) != 2 or any(t.dtype is not torch.uint8 or t.dim() != 2 for t in x):
        raise ValueError("rows in 8 bits are a pair of uint8 matrices, codes and scales")
    if cols is None:
        cols = x[0].shape[1]
        scales = -(-cols // 32)
    if x[0].shape[1] != cols or x[1].shape != (x[0].shape[0], scales):
        raise ValueError(f"codes {list(x[0].shape)} and scales {list(x[1].shape)} are not [R, {cols}] and [R, {scales}]")
    return x[0].contiguous(), x[1].contiguous()


def quantize_mx8(src: torch.Tensor) -> Kept:
    """MXFP8 codes (uint8 [R, C]) and scales (uint8 [R, ceil(C/32)]) of a bf16, fp16 or fp32 matrix of any
    width along its last axis (moe_quantize_mx8).  Codes carry no gradient: a source that requires one is
    refused (``detach`` it, or call under no_grad)."""
    if src.requires_grad and torch.is_grad_enabled():
        raise ValueError("the source requires a gradient, and MXFP8 codes have none: detach it")
    if src.dim() != 2:
        raise ValueError(f"expected a matrix, got {src.dim()} dimensions")
    row_dtype(src.dtype)
    device_index(src)
    return _quantize(src)


def _quantize(src: torch.Tensor) -> Kept:
    src, ld = _strided(src)
    rows, cols = src.shape
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=src.device)
    scales = torch.empty(rows, -(-cols // 32), dtype=torch.uint8, device=src.device)
    on_device(src.get_device(), M.moe_quantize_mx8, src.data_ptr(), ROW_DTYPES[src.dtype], rows, cols, ld,
              codes.data_ptr(), scales.data_ptr())
    return codes, scales


def dequantize_mx8(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of :func:`quantize_mx8`'s codes [R, C] (moe_dequantize_mx8)."""
    dt = row_dtype(dtype)
    codes, scales = _kept((codes, scales))
    dev = device_index(codes, scales)
    rows, cols = codes.shape
    out = torch.empty(rows, cols, dtype=dtype, device=codes.device)
    on_device(dev, M.moe_dequantize_mx8, codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), dt, cols)
    return out


def linear_backward(dy: torch.Tensor, x: Union[torch.Tensor, Kept, None], w: Optional[torch.Tensor],
                    offsets: Optional[torch.Tensor] = None, need_x: bool = True, need_w: bool = True,
                    w_dtype: Optional[torch.dtype] = None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of :func:`linear` from dy [R, N]: (dx [R, K] or None, dw [E, N, K], without offsets [N, K], or None).

    dx takes w and is zero in rows of no expert; dw takes x [R, K], or its codes and scales
    (:func:`quantize_mx8`), and is zero for an expert without rows.  Each may be None where its gradient is not
    needed.  dw is of dy's type or float32 (``w_dtype``)."""
    if dy.dtype not in _PRODUCT_DTYPES:
        raise ValueError(f"expected bfloat16 or float16 gradients, got {dy.dtype}")
    if dy.dim() != 2:
        raise ValueError(f"expected gradients [R, N], got {list(dy.shape)}")
    w_dtype = w_dtype or dy.dtype
    if w_dtype not in (dy.dtype, torch.float32):
        raise ValueError(f"the gradient of the weights is {dy.dtype} or float32, not {w_dtype}")
    if (need_x and w is None) or (need_w and x is None):
        raise ValueError("the rows' gradient takes the weights, the weights' gradient the rows")
    rows, n = dy.shape
    mats = k = None
    if need_x:
        mats, wn, k = _check_weights(w, offsets, dy.dtype)
        if wn != n:
            raise ValueError(f"expected gradients [R, {wn}], got {list(dy.shape)}")
    elif offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError(f"offsets must be int32 [E + 1], got {list(offsets.shape)}")
        mats = offsets.numel() - 1
    else:
        mats = 1
    offsets = _check_offsets(offsets, mats)
    codes = scales = None
    if not need_w:
        x = None
    else:
        if _is_kept(x):
            codes, scales = _kept(x)
            x, shape = None, codes.shape
        elif x.dtype != dy.dtype or x.dim() != 2:
            raise ValueError(f"expected rows [R, K] of type {dy.dtype}, got {x.dtype} {list(x.shape)}")
        else:
            shape = x.shape
        if shape[0] != rows or (need_x and shape[1] != k):
            raise ValueError(f"expected rows [{rows}, {k if need_x else 'K'}], got {list(shape)}")
        k = shape[1]
    if not (need_x or need_w):
        return None, None
    w = w if need_x else None
    device_index(dy, w, x, codes, scales, offsets)
    return _linear_back(dy, x, codes, scales, w, offsets, mats, n, k, need_x, need_w, w_dtype)


def _linear_back(dy, x, codes, scales, w, offsets, mats, n, k, need_x, need_w, w_dtype):
    rows, device = dy.shape[0], dy.device
    dy, ld_dy = _rows(dy)
    x, ld_x = (None, 0) if x is None else _rows(x)
    w = None if w is None else _dense(w)
    dt, w_dt = ROW_DTYPES[dy.dtype], ROW_DTYPES[w_dtype]
    dx = torch.empty(rows, k, dtype=dy.dtype, device=device) if need_x else None
    dw = torch.empty((n, k) if offsets is None else (mats, n, k), dtype=w_dtype, device=device) if need_w else None
    need = _backward_bytes(dt, rows, ld_dy, ld_x, mats, offsets is not None, n, k, need_x, k, need_w, w_dt)
    ws = _scratch(need, dy)
    on_device(dy.get_device(), M.moe_linear_rows_backward, dy.data_ptr(), dt, rows, ld_dy, _ptr(x), ld_x, _ptr(codes), _ptr(scales),
              _ptr(w), mats, _ptr(offsets), n, k, _ptr(dx), k, _ptr(dw), w_dt, _ptr(ws), need)
    return dx, dw


def _check_checkpoint(checkpoint: Optional[str]) -> bool:
    if checkpoint not in (None, "mx8"):
        raise ValueError(f"checkpoint is None (rows are kept as they are) or 'mx8', not {checkpoint!r}")
    return checkpoint is not None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, eight):
        need_x, need_w = x.requires_grad, w.requires_grad
        y = _linear(x, w, offsets)
        ctx.sizes = (1, *w.shape) if offsets is None else w.shape
        offsets = None if offsets is None else offsets.contiguous()
        kept = () if not need_w else _quantize(x) if eight else (x,)
        ctx.save_for_backward(w if need_x else None, offsets, *kept)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w, offsets, *kept = ctx.saved_tensors
        # (what came through the forward pass needs no more checks: in the thread that
        # runs backward passes Python takes several times as long)
        need_x, need_w = ctx.needs_input_grad[:2]
        x, codes, scales = (*kept, None, None) if len(kept) == 1 else (None, *kept) if kept else (None, None, None)
        dx, dw = _linear_back(dy, x if need_w else None, codes, scales, w if need_x else None, offsets, *ctx.sizes, need_x, need_w,
                              dy.dtype)
        return dx, dw, None, None


def linear(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor] = None,
           checkpoint: Optional[str] = None) -> torch.Tensor:
    """Rows times the matrix of their expert, y [R, N] of x's type (bfloat16 or float16), sums in fp32.

    x [R, K]; w [N, K], or [E, N, K] with ``offsets`` int32 [E+1]: rows offsets[e] .. offsets[e+1]-1 take
    matrix e (:func:`.tokens.sort_tokens`); rows of no expert give zeros.  Differentiable in x and w.
    ``checkpoint="mx8"`` keeps x for w's gradient in 8 bits (where w requires one).
    """
    eight = _check_checkpoint(checkpoint)
    if not (torch.is_grad_enabled() and (x.requires_grad or w.requires_grad)):
        return _linear(x, w, offsets)
    return _Linear.apply(x, w, offsets, eight)


def _swiglu(h: torch.Tensor, keep: bool) -> Tuple[torch.Tensor, Optional[Kept]]:
    if h.dim() != 2 or h.shape[1] % 2:
        raise ValueError(f"expected [R, 2 d_ff], got {list(h.shape)}")
    dt = row_dtype(h.dtype)
    dev = device_index(h)
    h, ld = _strided(h)
    rows, f = h.shape[0], h.shape[1] // 2
    a = torch.empty(rows, f, dtype=h.dtype, device=h.device)
    codes = scales = None
    if keep:
        codes = torch.empty(rows, 2 * f, dtype=torch.uint8, device=h.device)
        scales = torch.empty(rows, 2 * -(-f // 32), dtype=torch.uint8, device=h.device)
    on_device(dev, M.moe_swiglu, h.data_ptr(), dt, rows, f, ld, a.data_ptr(), f, _ptr(codes), _ptr(scales))
    return a, (codes, scales) if keep else None


def swiglu_backward(da: torch.Tensor, h: Union[torch.Tensor, Kept],
                    need_a: bool = False) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of :func:`swiglu`: dh [R, 2 d_ff] from da [R, d_ff] and h, or h's codes and scales as
    ``swiglu_keep`` gives them; with ``need_a`` also the activation of that h, else None."""
    row_dtype(da.dtype)
    if da.dim() != 2:
        raise ValueError(f"expected gradients [R, d_ff], got {list(da.shape)}")
    rows, f = da.shape
    codes = scales = None
    if _is_kept(h):
        codes, scales = _kept(h, 2 * f, 2 * -(-f // 32))
        h, h_rows = None, codes.shape[0]
    else:
        if h.dtype != da.dtype or h.dim() != 2 or h.shape[1] != 2 * f:
            raise ValueError(f"expected h [R, {2 * f}] of type {da.dtype}, got {h.dtype} {list(h.shape)}")
        h_rows = h.shape[0]
    if h_rows != rows:
        raise ValueError(f"{rows} rows of gradients for {h_rows} rows")
    device_index(da, h, codes, scales)
    return _swiglu_back(da, h, codes, scales, need_a)


def _swiglu_back(da, h, codes, scales, need_a):
    rows, f = da.shape
    da, ld_da = _strided(da)
    h, ld_h = (None, 0) if h is None else _strided(h)
    dh = torch.empty(rows, 2 * f, dtype=da.dtype, device=da.device)
    a = torch.empty(rows, f, dtype=da.dtype, device=da.device) if need_a else None
    on_device(da.get_device(), M.moe_swiglu_backward, da.data_ptr(), ROW_DTYPES[da.dtype], rows, f, ld_da, _ptr(h), ld_h, _ptr(codes), _ptr(scales),
              dh.data_ptr(), 2 * f, _ptr(a), f)
    return dh, a


def swiglu_keep(h: torch.Tensor) -> Tuple[torch.Tensor, Kept]:
    """The activation of h [R, 2 d_ff] and, from the same reading, h in 8 bits for :func:`swiglu_backward`:
    codes [R, 2 d_ff], scales [R, 2 ceil(d_ff/32)] (blocks do not reach over the halves).  No gradient."""
    if h.requires_grad and torch.is_grad_enabled():
        raise ValueError("h requires a gradient, and this has none: detach it, or call swiglu")
    return _swiglu(h, True)


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, eight):
        a, kept = _swiglu(h, eight)
        ctx.save_for_backward(*(kept if eight else (h,)))
        return a

    @staticmethod
    @once_differentiable
    def backward(ctx, da):
        kept = ctx.saved_tensors
        h, codes, scales = (*kept, None, None) if len(kept) == 1 else (None, *kept)
        return _swiglu_back(da, h, codes, scales, False)[0], None


def swiglu(h: torch.Tensor, checkpoint: Optional[str] = None) -> torch.Tensor:
    """The gated activation, silu(g) * u [R, d_ff] of h = [g, u] [R, 2 d_ff] (bf16, fp16 or fp32), computed in
    fp32.  Differentiable; ``checkpoint="mx8"`` keeps h for the gradient in 8 bits."""
    eight = _check_checkpoint(checkpoint)
    if not (torch.is_grad_enabled() and h.requires_grad):
        return _swiglu(h, False)[0]
    return _Swiglu.apply(h, eight)


class _Mlp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate_up, w_down, offsets, eight):
        need_x, need_gu, need_dn = x.requires_grad, w_gate_up.requires_grad, w_down.requires_grad
        h = _linear(x, w_gate_up, offsets)
        a, kept_h = _swiglu(h, eight)
        y = _linear(a, w_down, offsets)
        kept_x = () if not need_gu else _quantize(x) if eight else (x,)
        ctx.eight = eight
        # a is not kept: the backward pass has it again from h
        ctx.save_for_backward(w_gate_up if need_x else None, w_down if need_x or need_gu else None, offsets,
                              *(kept_h if eight else (h,)), *kept_x)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w_gate_up, w_down, offsets, *kept = ctx.saved_tensors
        h, x = (kept[:2], kept[2:]) if ctx.eight else (kept[0], kept[1] if len(kept) > 1 else None)
        need_x, need_gu, need_dn = ctx.needs_input_grad[:3]
        h_width = (h[0] if ctx.eight else h).shape[1]
        da = None
        if need_x or need_gu:
            da, _ = linear_backward(dy, None, w_down, offsets, True, False)
        # (where only w_down has a gradient, a is all that is taken of this)
        dh, a = swiglu_backward(dy.new_zeros(dy.shape[0], h_width // 2) if da is None else da, h, need_dn)
        dw_dn = linear_backward(dy, a, None, offsets, False, True)[1] if need_dn else None
        del a, da
        dx, dw_gu = linear_backward(dh, x or None if ctx.eight else x, w_gate_up, offsets, need_x, need_gu)
        return dx, dw_gu, dw_dn, None, None


def mlp(x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, offsets: Optional[torch.Tensor] = None,
        checkpoint: Optional[str] = None) -> torch.Tensor:
    """The experts' network on rows sorted by expert: linear(swiglu(linear(x, w_gate_up)), w_down), y [R, K].

    x [R, K], w_gate_up [E, 2 d_ff, K] (gate's rows first), w_down [E, K, d_ff], ``offsets`` as in
    :func:`linear`.  Differentiable in x and the weights.  Of the rows the backward pass keeps x and the
    activation's input, not its result; with ``checkpoint="mx8"`` both in 8 bits: K + 2 d_ff codes and
    (K + 2 d_ff)/32 scales a row."""
    eight = _check_checkpoint(checkpoint)
    if w_gate_up.dim() < 2 or w_down.dim() < 2 or w_gate_up.shape[-2] != 2 * w_down.shape[-1] or w_gate_up.shape[:-2] != w_down.shape[:-2]:
        raise ValueError(f"weights {list(w_gate_up.shape)} and {list(w_down.shape)} are not [E, 2 d_ff, K] and [E, M, d_ff]")
    if not (torch.is_grad_enabled() and (x.requires_grad or w_gate_up.requires_grad or w_down.requires_grad)):
        return _linear(_swiglu(_linear(x, w_gate_up, offsets), False)[0], w_down, offsets)
    return _Mlp.apply(x, w_gate_up, w_down, offsets, eight)
