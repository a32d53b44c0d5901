"""Torch-facing convenience wrapper: device buffers from PyTorch, every step of
the layer in the HIP library (through :mod:`.mxmoe`)."""

from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import mxmoe as M


@dataclass
class DeviceWeights:
    """MXFP4 expert weights (packed tile order, one flat row per expert, or
    canonical [E, N, K/2] codes and [E, N, K/32] scales, as ``layout`` says)
    and router parameters resident on one GPU."""
    gu_codes: torch.Tensor    # uint8 [E, d_ff*d]
    gu_scales: torch.Tensor   # uint8 [E, moe_packed_scale_bytes(2 d_ff, d)]
    dn_codes: torch.Tensor    # uint8 [E, d*d_ff/2]
    dn_scales: torch.Tensor   # uint8 [E, moe_packed_scale_bytes(d, d_ff)]
    sgu_codes: Optional[torch.Tensor]
    sgu_scales: Optional[torch.Tensor]
    sdn_codes: Optional[torch.Tensor]
    sdn_scales: Optional[torch.Tensor]
    router_w: torch.Tensor    # float32 [E, d]
    router_b: Optional[torch.Tensor]
    layout: int = M.MOE_WEIGHTS_PACKED

    def abi(self) -> M.MoeWeights:
        p = lambda t: (t.data_ptr() if t is not None else None)
        return M.MoeWeights(p(self.gu_codes), p(self.gu_scales), p(self.dn_codes),
                            p(self.dn_scales), p(self.sgu_codes), p(self.sgu_scales),
                            p(self.sdn_codes), p(self.sdn_scales), p(self.router_w),
                            p(self.router_b), self.layout)


class MoeLayer:
    """One MoE layer on the current CUDA/HIP device."""

    def __init__(self, d_model: int, d_ff: int, num_experts: int, top_k: int, num_shared: int,
                 max_tokens: int, weights: DeviceWeights, flags: int = 0):
        self.shape = dict(d_model=d_model, d_ff=d_ff, num_experts=num_experts, top_k=top_k,
                          num_shared=num_shared, max_tokens=max_tokens, flags=flags)
        self.plan = M.moe_plan(d_model, d_ff, num_experts, top_k, num_shared, max_tokens, flags)
        self.weights = weights
        self._wabi = weights.abi()
        self._ws: Optional[torch.Tensor] = None

    def __del__(self):
        try:
            M.moe_plan_destroy(self.plan)
        except Exception:
            pass

    def workspace_bytes(self, num_tokens: int) -> int:
        return M.moe_workspace_bytes(self.plan, num_tokens)

    def workspace(self, num_tokens: int, device=None) -> torch.Tensor:
        need = self.workspace_bytes(num_tokens)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 256), dtype=torch.uint8,
                                   device=device or self.weights.router_w.device)
        return self._ws

    def forward(self, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                taps: Optional[Dict[str, torch.Tensor]] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x: bfloat16 [T, d] on the device -> y bfloat16 [T, d]."""
        assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 2
        t = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        ws = workspace if workspace is not None else self.workspace(t, x.device)
        tp = None
        if taps:
            tp = M.MoeTaps(**{k: v.data_ptr() for k, v in taps.items()})
        M.moe_forward(self.plan, self._wabi, x.data_ptr(), t, y.data_ptr(), ws.data_ptr(),
                      ws.numel(), tp, torch.cuda.current_stream().cuda_stream)
        return y


def quantize_act(src: torch.Tensor):
    """MXFP8 codes and scales of a 2-D bf16/fp32 tensor along its last axis."""
    assert src.dim() == 2 and src.stride(1) == 1
    rows, cols = src.shape
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=src.device)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=src.device)
    dt = M.MOE_SRC_FP32 if src.dtype == torch.float32 else M.MOE_SRC_BF16
    assert src.dtype in (torch.float32, torch.bfloat16)
    M.moe_quantize_act(src.data_ptr(), dt, rows, cols, src.stride(0), codes.data_ptr(),
                       scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
    return codes, scales


# element types of plain matrices taken by the functions below
ROW_DTYPES = {torch.bfloat16: M.MOE_SRC_BF16, torch.float32: M.MOE_SRC_FP32, torch.float16: M.MOE_SRC_FP16}


def row_dtype(dtype: torch.dtype) -> int:
    dt = ROW_DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"expected bfloat16, float16 or float32, got {dtype}")
    return dt


def device_index(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The GPU that every tensor is on (a call's launches go to its current stream).
    A tensor with a forward-mode tangent is refused: the kernels see values only,
    and their outputs would come without one."""
    if forward_ad._current_level >= 0:  # (inside a dual_level: elsewhere there are no tangents)
        for t in (first, *others):
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("a tensor has a forward-mode tangent, and there is no forward-mode derivative here")
    if not first.is_cuda:
        raise ValueError(f"expected tensors on a GPU, got one on {first.device}")
    index = first.get_device()
    for t in others:
        if t is not None and (t.get_device() != index or not t.is_cuda):
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    return index


def in_memory(t: torch.Tensor) -> torch.Tensor:
    """t, with its values where its address says: a conjugated view, or its
    imaginary part, shares the memory of the values before."""
    return t.resolve_conj().resolve_neg() if t.is_neg() or t.is_conj() else t


def on_device(index: int, call, *args) -> None:
    """call(*args, stream) with GPU ``index`` current and its current stream.  A few
    small calls are bound by the host: the device is switched only if it has to be."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        call(*args, stream)
    else:
        with torch.cuda.device(index):
            call(*args, stream)


def _mx4_operand(codes: torch.Tensor, scales: torch.Tensor, what: str, dims: int):
    """Contiguous canonical codes [..., K/2] and scales [..., K/32]; -> (codes, scales, K)"""
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError(f"{what}: codes and scales must be uint8")
    cs, ss = codes.shape, scales.shape
    if len(cs) != dims or len(ss) != dims or cs[:-1] != ss[:-1] or cs[-1] != 16 * ss[-1]:
        raise ValueError(f"{what}: codes {tuple(cs)} and scales {tuple(ss)} are not [..., K/2] and [..., K/32]")
    if not codes.is_contiguous():
        codes = codes.contiguous()
    if not scales.is_contiguous():
        scales = scales.contiguous()
    if codes.data_ptr() % 16:
        codes = codes.clone()
    return codes, scales, 32 * ss[-1]


def quantize_mx4(src: torch.Tensor):
    """MXFP4 codes (uint8 [rows, cols/2]) and scales (uint8 [rows, cols/32]) of a
    2-D bf16, fp16 or fp32 tensor along its last axis, in the canonical form of
    the expert weights (moe_quantize_mx4).  Codes carry no gradient: a source
    that requires one is refused (``detach`` it, or call under no_grad)."""
    if src.requires_grad and torch.is_grad_enabled():
        raise ValueError("the source requires a gradient, and MXFP4 codes have none: detach it")
    if src.dim() != 2:
        raise ValueError(f"expected a matrix, got {src.dim()} dimensions")
    dt = row_dtype(src.dtype)
    dev = device_index(src)
    rows, cols = src.shape
    if cols % 32:
        raise ValueError(f"columns ({cols}) must be a multiple of 32")
    src = in_memory(src)
    ld, step = src.stride()
    if cols and (step != 1 or ld < cols):
        src = src.contiguous()
        ld = cols
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=src.device)
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=src.device)
    on_device(dev, M.moe_quantize_mx4, src.data_ptr(), dt, rows, cols, max(ld, cols), codes.data_ptr(),
              scales.data_ptr())
    return codes, scales


def dequantize_mx4(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of a canonical MXFP4 matrix [rows, K/2], [rows, K/32] (moe_dequantize_mx4)."""
    dt = row_dtype(dtype)
    dev = device_index(codes, scales)
    codes, scales, cols = _mx4_operand(codes, scales, "matrix", 2)
    rows = codes.shape[0]
    out = torch.empty(rows, cols, dtype=dtype, device=codes.device)
    on_device(dev, M.moe_dequantize_mx4, codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), dt, cols)
    return out


def linear_mx4(codes: torch.Tensor, scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows times weights, both MXFP4 in canonical form, fp32 accumulation (moe_linear_mx4).

    codes [R, K/2], scales [R, K/32]; w_codes [N, K/2], w_scales [N, K/32], or
    with a leading axis of matrices [E, N, ...] and ``offsets`` int32 [E+1]:
    rows offsets[e] .. offsets[e+1]-1 take matrix e.  Rows outside every range
    are left as they were in ``out``; without ``out`` they are undefined.
    ``dtype`` is the result's: ``out``'s, or bfloat16 where neither is given.
    No gradient: the product is for inference, and ``out`` may not require one
    (except under no_grad).
    """
    if out is not None and out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out requires a gradient, and the product has none")
    if out is not None and dtype is not None and dtype != out.dtype:
        raise ValueError(f"the result is to be {dtype}, and out is {out.dtype}")
    grouped = offsets is not None
    dev = device_index(codes, scales, w_codes, w_scales, offsets, out)
    codes, scales, k = _mx4_operand(codes, scales, "rows", 2)
    w_codes, w_scales, wk = _mx4_operand(w_codes, w_scales, "weights", 3 if grouped else 2)
    if k != wk:
        raise ValueError(f"rows have K = {k}, weights K = {wk}")
    mats, n = (w_codes.shape[0] if grouped else 1), w_codes.shape[-2]
    at = None
    if grouped:
        if offsets.dtype is not torch.int32 or offsets.shape != (mats + 1,):
            raise ValueError(f"offsets must be int32 [{mats + 1}]")
        if not offsets.is_contiguous():
            offsets = offsets.contiguous()
        at = offsets.data_ptr()
    rows = codes.shape[0]
    given = out is not None
    if not given:
        out, ld = torch.empty(rows, n, dtype=dtype or torch.bfloat16, device=codes.device), n
    else:
        if out.is_neg():
            raise ValueError("out is a lazily negated view")
        ld = out.stride(0) if out.dim() == 2 and rows > 1 else n
        if out.shape != (rows, n) or (n > 1 and out.stride(1) != 1) or ld < n:
            raise ValueError(f"out must be [{rows}, {n}] with dense rows")
    on_device(dev, M.moe_linear_mx4, codes.data_ptr(), scales.data_ptr(), rows, w_codes.data_ptr(),
              w_scales.data_ptr(), mats, at, n, k, out.data_ptr(), row_dtype(out.dtype), ld)
    if given:
        # autograd learns of the write: what it saved of out before is no longer there
        increment_version(out)
    return out
