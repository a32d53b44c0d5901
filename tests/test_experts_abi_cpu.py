"""Argument checks of the 16-bit products, of activations in 8 bits and of the
gated activation, on the host (no GPU): every refusal comes before a device
call, with the documented status."""

import os

import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from mxfp4_expert_grouped_amd import mxmoe
    if not os.path.exists(mxmoe.LIB_PATH):
        from mxfp4_expert_grouped_amd import build
        build.build()
    mxmoe.load_library()
    return mxmoe


FAKE = 1 << 20  # never dereferenced: the calls fail their checks, or have nothing to do
INV, UNS, WSP, DEV = 1, 2, 3, 4
BF16, FP32, FP16 = 0, 1, 2


def refused(M, fn, base, over, status):
    args = {**base, **over}
    with pytest.raises(M.MoeError) as ei:
        fn(*args.values())
    assert ei.value.status == status, (over, ei.value)
    assert ei.value.detail


FORWARD = dict(x=FAKE, dt=BF16, rows=4, ld_x=16, w=FAKE, mats=2, offsets=FAKE, n=8, k=16, y=FAKE, ld_y=8, ws=FAKE, bytes=1 << 40)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(dt=-1), INV), (dict(dt=FP32), UNS), (dict(rows=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV),
    (dict(mats=0), INV), (dict(mats=-1), INV), (dict(mats=2, offsets=None), INV), (dict(mats=1025), UNS), (dict(rows=(1 << 25) + 1), UNS),
    (dict(n=(1 << 20) + 1, ld_y=1 << 21), UNS), (dict(k=(1 << 20) + 1, ld_x=1 << 21), UNS), (dict(ld_x=15), INV), (dict(ld_y=7), INV),
    (dict(ld_x=(1 << 21) + 1), UNS), (dict(ld_y=(1 << 21) + 1), UNS), (dict(rows=1 << 25, n=1 << 20, ld_y=1 << 20), UNS),
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(x=FAKE + 8), INV), (dict(w=FAKE + 2), INV), (dict(y=FAKE + 1), INV),
    (dict(offsets=FAKE + 2), INV),
])
def test_linear_rows(M, over, status):
    refused(M, M.moe_linear_rows, FORWARD, over, status)


BACKWARD = dict(dy=FAKE, dt=FP16, rows=4, ld_dy=8, x=FAKE, ld_x=16, codes=None, scales=None, w=FAKE, mats=2, offsets=FAKE, n=8, k=16,
                dx=FAKE, ld_dx=16, dw=FAKE, dw_dt=FP16, ws=FAKE, bytes=1 << 40)
CODES = dict(x=None, ld_x=0, codes=FAKE, scales=FAKE)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(dt=FP32), UNS), (dict(rows=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV), (dict(mats=0), INV),
    (dict(offsets=None), INV), (dict(mats=1025), UNS), (dict(rows=(1 << 25) + 1), UNS), (dict(ld_dy=7), INV), (dict(ld_x=15), INV),
    (dict(ld_dx=15), INV), (dict(ld_dy=(1 << 21) + 1), UNS), (dict(ld_x=(1 << 21) + 1), UNS), (dict(ld_dx=(1 << 21) + 1), UNS),
    (dict(dw_dt=BF16), INV), (dict(dw_dt=3), INV), (dict(dy=None), INV), (dict(x=None), INV), (dict(w=None), INV),
    (dict(dy=FAKE + 8), INV), (dict(x=FAKE + 8), INV), (dict(w=FAKE + 8), INV), (dict(dx=FAKE + 1), INV), (dict(dw=FAKE + 1), INV),
    (dict(dw=FAKE + 4, dw_dt=FP32), INV), (dict(offsets=FAKE + 1), INV), (dict(codes=FAKE, scales=FAKE), INV), (dict(codes=FAKE), INV),
    (dict(CODES, scales=None), INV), (dict(CODES, ld_x=16), INV), (dict(ld_x=0), INV),
    (dict(dx=None, mats=1024, n=1 << 20, k=1 << 20, ld_dy=1 << 20, ld_x=1 << 20), UNS),
])
def test_linear_rows_backward(M, over, status):
    refused(M, M.moe_linear_rows_backward, BACKWARD, over, status)


def test_workspaces(M):
    # widths that are no multiples of 8 are laid out, x from 8 bits too
    fwd = lambda rows, ld, n, k, mats=2: M.moe_linear_rows_workspace_bytes(BF16, rows, ld, mats, 1, n, k, n)  # noqa: E731
    back = lambda ld_dy, ld_x, n, k, dx=1, dw=1, rows=4000, dt=BF16: M.moe_linear_rows_backward_workspace_bytes(  # noqa: E731
        BF16, rows, ld_dy, ld_x, 2, 1, n, k, dx, k, dw, dt)
    assert fwd(40000, 512, 256, 512) == 0
    assert fwd(40000, 511, 256, 511) >= 2 * 512 * (40000 + 2 * 256)
    assert 2 * 512 * 40000 <= fwd(40000, 513, 256, 512) < 2 * 512 * (40000 + 256)
    assert back(2048, 1024, 2048, 1024) == 0
    assert back(2048, 0, 2048, 1024) >= 2 * 1024 * 4000
    assert back(2048, 0, 2048, 1024, dw=0) == 0
    assert back(2047, 1023, 2047, 1023) >= 2 * (2048 * 4000 + 1024 * 4000 + 2 * 2047 * 1024)
    assert back(2048, 1023, 2048, 1023, dx=0, dt=FP32) >= 4 * 2 * 2048 * 1024  # fp32 rows of no whole pieces are joined
    need = fwd(40000, 511, 256, 511)
    base = {**FORWARD, "rows": 40000, "ld_x": 511, "k": 511, "n": 256, "ld_y": 256}
    for over in (dict(ws=None), dict(bytes=need - 1), dict(ws=FAKE + 16)):
        refused(M, M.moe_linear_rows, base, over, WSP)
    base = {**BACKWARD, "rows": 4000, "ld_dy": 7, "n": 7}
    for over in (dict(ws=None), dict(bytes=8), dict(ws=FAKE + 128)):
        refused(M, M.moe_linear_rows_backward, base, over, WSP)
    for bad in (lambda: M.moe_linear_rows_workspace_bytes(FP32, 4, 8, 1, 0, 8, 8, 8),
                lambda: M.moe_linear_rows_workspace_bytes(BF16, 4, 7, 1, 0, 8, 8, 8),
                lambda: M.moe_linear_rows_workspace_bytes(BF16, 4, 8, 2, 0, 8, 8, 8),
                lambda: M.moe_linear_rows_backward_workspace_bytes(BF16, 4, 8, 7, 1, 0, 8, 8, 1, 8, 1, BF16)):
        with pytest.raises(M.MoeError):
            bad()


def test_products_of_nothing(M):
    M.moe_linear_rows(None, BF16, 0, 16, None, 2, FAKE, 8, 16, None, 8, None, 0)
    M.moe_linear_rows(None, BF16, 4, 16, None, 2, FAKE, 0, 16, None, 0, None, 0)
    for over in (dict(dx=None, dw=None), dict(k=0, ld_x=0, ld_dx=0, x=None), dict(rows=0, dw=None, dy=None, x=None, w=None),
                 dict(n=0, dx=None, dw_dt=FP16)):
        M.moe_linear_rows_backward(*{**BACKWARD, **over}.values())


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(dt=-1), INV), (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(ld=63), INV), (dict(plain=None), INV),
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(plain=FAKE + 1), INV), (dict(plain=FAKE + 2, dt=FP32), INV),
    (dict(rows=(1 << 40) + 1), UNS), (dict(cols=(1 << 28) + 1, ld=1 << 29), UNS), (dict(ld=1 << 41), UNS),
])
def test_mx8_conversions(M, over, status):
    base = dict(plain=FAKE, dt=BF16, rows=4, cols=64, ld=64, codes=FAKE, scales=FAKE)
    refused(M, M.moe_quantize_mx8, base, over, status)
    refused(M, M.moe_dequantize_mx8, {n: base[n] for n in ("codes", "scales", "rows", "cols", "plain", "dt", "ld")}, over, status)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(rows=-1), INV), (dict(f=-1), INV), (dict(ld_h=31), INV), (dict(ld_a=15), INV), (dict(h=None), INV),
    (dict(a=None), INV), (dict(codes=FAKE), INV), (dict(scales=FAKE), INV), (dict(h=FAKE + 1), INV), (dict(a=FAKE + 1), INV),
    (dict(rows=(1 << 40) + 1), UNS), (dict(f=(1 << 28) + 1, ld_h=1 << 30, ld_a=1 << 30), UNS), (dict(ld_h=1 << 41), UNS),
])
def test_swiglu(M, over, status):
    refused(M, M.moe_swiglu, dict(h=FAKE, dt=BF16, rows=4, f=16, ld_h=32, a=FAKE, ld_a=16, codes=None, scales=None), over, status)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(rows=-1), INV), (dict(f=-1), INV), (dict(ld_da=15), INV), (dict(ld_h=31), INV), (dict(ld_dh=31), INV),
    (dict(ld_a=15), INV), (dict(da=None), INV), (dict(h=None), INV), (dict(dh=None), INV), (dict(codes=FAKE), INV), (dict(codes=FAKE, scales=FAKE), INV),
    (dict(h=None, codes=FAKE), INV), (dict(da=FAKE + 1), INV), (dict(h=FAKE + 1), INV), (dict(dh=FAKE + 1), INV), (dict(a=FAKE + 1), INV),
    (dict(ld_dh=1 << 41), UNS),
])
def test_swiglu_backward(M, over, status):
    refused(M, M.moe_swiglu_backward, dict(da=FAKE, dt=BF16, rows=4, f=16, ld_da=16, h=FAKE, ld_h=32, codes=None, scales=None, dh=FAKE,
                                           ld_dh=32, a=FAKE, ld_a=16), over, status)


def test_activations_of_nothing(M):
    M.moe_quantize_mx8(None, BF16, 0, 64, 64, None, None)
    M.moe_quantize_mx8(None, FP32, 4, 0, 0, None, None)
    M.moe_dequantize_mx8(None, None, 0, 64, None, FP16, 64)
    M.moe_swiglu(None, BF16, 0, 16, 32, None, 16, None, None)
    M.moe_swiglu_backward(None, BF16, 4, 0, 0, None, 0, None, None, None, 0, None, 0)


# ---- the torch forms


@pytest.fixture(scope="module")
def X():
    from mxfp4_expert_grouped_amd import experts
    return experts


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_torch_refusals(X):
    u8 = torch.uint8
    bad = [
        lambda: X.linear(t(4, 8, dtype=torch.float32), t(6, 8, dtype=torch.float32)), lambda: X.linear(t(4, 8), t(6, 8, dtype=torch.float16)),
        lambda: X.linear(t(4, 8), t(2, 6, 8)), lambda: X.linear(t(4, 8), t(6, 8), ints(2)), lambda: X.linear(t(4, 7), t(6, 8)),
        lambda: X.linear(t(4), t(6, 8)), lambda: X.linear(t(4, 8), t(2, 6, 8), ints(2)), lambda: X.linear(t(4, 8), t(2, 6, 8), ints(3).long()),
        lambda: X.linear(t(4, 8), t(2, 6, 8), ints(3, 1)), lambda: X.linear(t(4, 8), t(6, 8), checkpoint="fp8"),
        lambda: X.linear(t(4, 8), t(6, 8), checkpoint=True),
        lambda: X.linear_backward(t(4, 6), t(4, 8), t(5, 8)), lambda: X.linear_backward(t(4, 6), t(3, 8), t(6, 8)),
        lambda: X.linear_backward(t(4, 6), t(4, 7), t(6, 8)), lambda: X.linear_backward(t(4, 6), None, t(6, 8)),
        lambda: X.linear_backward(t(4, 6), t(4, 8), None), lambda: X.linear_backward(t(4, 6, dtype=torch.float32), t(4, 8), t(6, 8)),
        lambda: X.linear_backward(t(4, 6), t(4, 8, dtype=torch.float16), t(6, 8)), lambda: X.linear_backward(t(4, 6), t(4, 8), t(6, 8), w_dtype=torch.float16),
        lambda: X.linear_backward(t(4, 6), t(4, 8), None, ints(1), need_x=False), lambda: X.linear_backward(t(4, 6), t(4, 8), None, ints(3, 2), need_x=False),
        lambda: X.linear_backward(t(4, 6), (t(4, 8), t(4, 1)), t(6, 8)), lambda: X.linear_backward(t(4, 6), (t(4, 40, dtype=u8), t(4, 1, dtype=u8)), None, need_x=False),
        lambda: X.linear_backward(t(4, 6), (t(3, 8, dtype=u8), t(3, 1, dtype=u8)), t(6, 8)),
        lambda: X.quantize_mx8(t(4)), lambda: X.quantize_mx8(ints(4, 4)), lambda: X.quantize_mx8(t(4, 4).requires_grad_()),
        lambda: X.dequantize_mx8(t(4, 33, dtype=u8), t(4, 1, dtype=u8)),
        lambda: X.swiglu(t(4, 7)), lambda: X.swiglu(t(8)), lambda: X.swiglu(ints(4, 8)), lambda: X.swiglu(t(4, 8), checkpoint="x"),
        lambda: X.swiglu_keep(t(4, 8).requires_grad_()), lambda: X.swiglu_backward(t(4, 4), t(4, 6)), lambda: X.swiglu_backward(t(4, 4), t(3, 8)),
        lambda: X.swiglu_backward(t(4, 4), t(4, 8, dtype=torch.float16)), lambda: X.swiglu_backward(t(4, 4), (t(4, 8, dtype=u8), t(4, 1, dtype=u8))),
        lambda: X.mlp(t(4, 8), t(6, 8), t(8, 4)), lambda: X.mlp(t(4, 8), t(2, 6, 8), t(3, 8, 3), ints(3)), lambda: X.mlp(t(4, 8), t(6, 8), t(8, 3), checkpoint="y"),
    ]
    for call in bad:
        with pytest.raises((ValueError, NotImplementedError)) as ei:
            call()
        assert "GPU" not in str(ei.value)


def test_torch_forms_need_a_gpu(X):
    u8 = torch.uint8
    for call in (lambda: X.linear(t(4, 8), t(6, 8)), lambda: X.linear(t(4, 8), t(2, 6, 8), ints(3)), lambda: X.linear_backward(t(4, 6), t(4, 8), t(6, 8)),
                 lambda: X.quantize_mx8(t(4, 4)), lambda: X.dequantize_mx8(t(4, 33, dtype=u8), t(4, 2, dtype=u8)), lambda: X.swiglu(t(4, 8)),
                 lambda: X.swiglu(t(4, 8).requires_grad_(), checkpoint="mx8"), lambda: X.swiglu_keep(t(4, 8)), lambda: X.swiglu_backward(t(4, 4), t(4, 8)),
                 lambda: X.mlp(t(4, 8), t(6, 8), t(8, 3)), lambda: X.linear(t(4, 8).requires_grad_(), t(6, 8), checkpoint="mx8")):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_forward_mode_tangent_is_refused(X):
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        dual = lambda *s: forward_ad.make_dual(torch.ones(s).bfloat16(), torch.ones(s).bfloat16())  # noqa: E731
        for call in (lambda: X.linear(dual(4, 8), t(6, 8)), lambda: X.linear(t(4, 8), dual(6, 8)), lambda: X.linear_backward(dual(4, 6), t(4, 8), t(6, 8)),
                     lambda: X.quantize_mx8(dual(4, 4)), lambda: X.swiglu(dual(4, 8)), lambda: X.swiglu_backward(t(4, 4), dual(4, 8)),
                     lambda: X.mlp(dual(4, 8), t(6, 8), t(8, 3))):
            with pytest.raises(NotImplementedError, match="tangent"):
                call()


def test_operands_without_dimensions_are_refused(X):
    u, dy = torch.zeros((), dtype=torch.uint8), t(2, 8)
    for call in (lambda: X.dequantize_mx8(u, u), lambda: X.linear_backward(dy, (), None, need_x=False),
                 lambda: X.linear_backward(dy, (u, u), None, need_x=False), lambda: X.swiglu_backward(dy, (u, u)),
                 lambda: X.mlp(dy, t(), t()), lambda: X.mlp(dy, t(8), t(4)), lambda: X.linear(dy, t())):
        with pytest.raises(ValueError):
            call()
