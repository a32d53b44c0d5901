"""Torch-facing convenience wrapper: device buffers from PyTorch, every step of
the layer in the HIP library (through :mod:`.mxmoe`)."""

from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, Optional

import torch

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
    if dtype not in ROW_DTYPES:
        raise ValueError(f"expected bfloat16, float16 or float32, got {dtype}")
    return ROW_DTYPES[dtype]


def check_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    """Every tensor on one GPU (the launches go to its current stream)."""
    if first.device.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got one on {first.device}")
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")


def stream_of(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _mx4_operand(codes: torch.Tensor, scales: torch.Tensor, what: str, dims: int):
    """Contiguous canonical codes [..., K/2] and scales [..., K/32]; -> (codes, scales, K)"""
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError(f"{what}: codes and scales must be uint8")
    if codes.dim() != dims or scales.dim() != dims or codes.shape[:-1] != scales.shape[:-1] \
            or codes.shape[-1] != 16 * scales.shape[-1]:
        raise ValueError(f"{what}: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} are not "
                         "[..., K/2] and [..., K/32]")
    codes, scales = codes.contiguous(), scales.contiguous()
    if codes.data_ptr() % 16:
        codes = codes.clone()
    return codes, scales, 32 * scales.shape[-1]


def quantize_mx4(src: torch.Tensor):
    """MXFP4 codes (uint8 [rows, cols/2]) and scales (uint8 [rows, cols/32]) of a
    2-D bf16, fp16 or fp32 tensor along its last axis, in the canonical form of
    the expert weights (moe_quantize_mx4)."""
    if src.dim() != 2:
        raise ValueError(f"expected a matrix, got {src.dim()} dimensions")
    dt = row_dtype(src.dtype)
    check_device(src)
    rows, cols = src.shape
    if cols % 32:
        raise ValueError(f"columns ({cols}) must be a multiple of 32")
    if cols and (src.stride(1) != 1 or src.stride(0) < cols):
        src = src.contiguous()
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=src.device)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=src.device)
    with torch.cuda.device(src.device):
        M.moe_quantize_mx4(src.data_ptr(), dt, rows, cols, max(src.stride(0), cols), codes.data_ptr(),
                           scales.data_ptr(), stream_of(src))
    return codes, scales


def dequantize_mx4(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of a canonical MXFP4 matrix [rows, K/2], [rows, K/32] (moe_dequantize_mx4)."""
    dt = row_dtype(dtype)
    check_device(codes, scales)
    codes, scales, cols = _mx4_operand(codes, scales, "matrix", 2)
    rows = codes.shape[0]
    out = torch.empty((rows, cols), dtype=dtype, device=codes.device)
    with torch.cuda.device(codes.device):
        M.moe_dequantize_mx4(codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), dt, cols,
                             stream_of(codes))
    return out


def linear_mx4(codes: torch.Tensor, scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows times weights, both MXFP4 in canonical form, fp32 accumulation (moe_linear_mx4).

    codes [R, K/2], scales [R, K/32]; w_codes [N, K/2], w_scales [N, K/32], or
    with a leading axis of matrices [E, N, ...] and ``offsets`` int32 [E+1]:
    rows offsets[e] .. offsets[e+1]-1 take matrix e.  Rows outside every range
    are left as they were in ``out``; without ``out`` they are undefined.
    No gradient: the product is for inference.
    """
    grouped = offsets is not None
    check_device(codes, scales, w_codes, w_scales, offsets, out)
    codes, scales, k = _mx4_operand(codes, scales, "rows", 2)
    w_codes, w_scales, wk = _mx4_operand(w_codes, w_scales, "weights", 3 if grouped else 2)
    if k != wk:
        raise ValueError(f"rows have K = {k}, weights K = {wk}")
    mats, n = (w_codes.shape[0] if grouped else 1), w_codes.shape[-2]
    if grouped and (offsets.dtype != torch.int32 or offsets.shape != (mats + 1,)):
        raise ValueError(f"offsets must be int32 [{mats + 1}]")
    rows = codes.shape[0]
    if out is None:
        out = torch.empty((rows, n), dtype=dtype, device=codes.device)
    elif out.shape != (rows, n) or (n and out.stride(1) != 1) or (rows > 1 and out.stride(0) < n):
        raise ValueError(f"out must be [{rows}, {n}] with dense rows")
    dt = row_dtype(out.dtype)
    with torch.cuda.device(codes.device):
        M.moe_linear_mx4(codes.data_ptr(), scales.data_ptr(), rows, w_codes.data_ptr(), w_scales.data_ptr(),
                         mats, offsets.contiguous().data_ptr() if grouped else None, n, k, out.data_ptr(), dt,
                         max(out.stride(0), n), stream_of(codes))
    return out
