"""Argument checks of the layer's standalone pieces, on the host (no GPU):
every refusal comes before a device call, with the documented status."""

import os

import pytest


@pytest.fixture(scope="module")
def M():
    from mxfp4_expert_grouped_amd import mxmoe
    if not os.path.exists(mxmoe.LIB_PATH):
        from mxfp4_expert_grouped_amd import build
        build.build()
    mxmoe.load_library()
    return mxmoe


FAKE = 1 << 20  # never dereferenced: the calls fail their checks, or have nothing to do
INV, UNS, WSP = 1, 2, 3


def refused(M, fn, base, over, status):
    args = dict(base)
    args.update(over)
    with pytest.raises(M.MoeError) as ei:
        fn(*args.values())
    assert ei.value.status == status, (over, ei.value)
    assert ei.value.detail


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(dt=-1), INV), (dict(rows=-1), INV), (dict(cols=-32), INV), (dict(cols=48), UNS),
    (dict(ld=32), INV), (dict(plain=None), INV), (dict(codes=None), INV), (dict(scales=None), INV),
    (dict(plain=FAKE + 1), INV), (dict(codes=FAKE + 2), INV), (dict(rows=(1 << 40) + 1), UNS),
    (dict(cols=1 << 31, ld=1 << 31), UNS), (dict(ld=1 << 41), UNS), (dict(plain=FAKE + 2, dt=1), INV),
])
def test_mx4_conversions(M, over, status):
    base = dict(plain=FAKE, dt=0, rows=4, cols=64, ld=64, codes=FAKE, scales=FAKE)
    refused(M, M.moe_quantize_mx4, base, over, status)
    back = {n: base[n] for n in ("codes", "scales", "rows", "cols", "plain", "dt", "ld")}
    refused(M, M.moe_dequantize_mx4, back, over, status)


def test_mx4_conversions_of_nothing(M):
    M.moe_quantize_mx4(None, 0, 0, 64, 64, None, None)
    M.moe_quantize_mx4(None, 2, 4, 0, 0, None, None)
    M.moe_dequantize_mx4(None, None, 0, 64, None, 1, 64)


def test_quantize_act_still_refuses_fp16(M):
    with pytest.raises(M.MoeError) as ei:
        M.moe_quantize_act(FAKE, M.MOE_SRC_FP16, 4, 64, 64, FAKE, FAKE)
    assert ei.value.status == INV


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(rows=-1), INV), (dict(n=-1), INV), (dict(k=0), INV), (dict(k=-32), INV), (dict(k=48), UNS),
    (dict(k=65536 + 32), UNS), (dict(mats=0), INV), (dict(mats=1025), UNS), (dict(mats=2, offsets=None), INV),
    (dict(n=(1 << 20) + 1, ld=1 << 21), UNS), (dict(rows=(1 << 25) + 1), UNS), (dict(ld=15), INV), (dict(ld=1 << 33), UNS),
    (dict(ac=None), INV), (dict(asc=None), INV), (dict(wc=None), INV), (dict(wsc=None), INV), (dict(y=None), INV),
    (dict(ac=FAKE + 8), INV), (dict(wc=FAKE + 4), INV), (dict(y=FAKE + 1), INV), (dict(offsets=FAKE + 2), INV),
    (dict(y=FAKE + 2, dt=1), INV),
])
def test_linear(M, over, status):
    base = dict(ac=FAKE, asc=FAKE, rows=4, wc=FAKE, wsc=FAKE, mats=2, offsets=FAKE, n=16, k=64, y=FAKE, dt=0, ld=16)
    refused(M, M.moe_linear_mx4, base, over, status)


def test_linear_of_nothing(M):
    M.moe_linear_mx4(None, None, 0, None, None, 1, None, 16, 64, None, 0, 16)
    M.moe_linear_mx4(None, None, 4, None, None, 1, None, 0, 64, None, 0, 0)


@pytest.mark.parametrize("over,status", [
    (dict(dt=2), INV), (dict(t=-1), INV), (dict(t=(1 << 20) + 1), INV), (dict(k=0), INV), (dict(k=33), INV), (dict(e=0), INV),
    (dict(e=1025), INV), (dict(ids=None), INV), (dict(off=None), INV), (dict(src=None), INV), (dict(tr=None), INV),
    (dict(ids=FAKE + 2), INV), (dict(ids=FAKE + 4, dt=1), INV), (dict(off=FAKE + 1), INV),
    (dict(t=100000), WSP), (dict(t=100000, ws=FAKE, bytes=1 << 10), WSP), (dict(t=100000, ws=FAKE + 16, bytes=1 << 30), WSP),
])
def test_sort_tokens(M, over, status):
    base = dict(ids=FAKE, dt=0, t=4, k=2, e=8, off=FAKE, src=FAKE, tr=FAKE, ws=None, bytes=0)
    refused(M, M.moe_sort_tokens, base, over, status)


def test_sort_tokens_workspace(M):
    assert M.moe_sort_tokens_workspace_bytes(0, 1, 1) == 0
    assert M.moe_sort_tokens_workspace_bytes(1, 32, 1024) == 0
    big = M.moe_sort_tokens_workspace_bytes(1 << 20, 32, 1024)
    assert 0 < M.moe_sort_tokens_workspace_bytes(8192, 16, 896) <= big <= (1 << 13) * 1024 * 4
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 33, 1), (1, 1, 0), (1, 1, 1025), ((1 << 20) + 1, 1, 1)):
        with pytest.raises(M.MoeError):
            M.moe_sort_tokens_workspace_bytes(*bad)


@pytest.mark.parametrize("over,status", [
    (dict(bytes=-1), INV), (dict(ldx=63), INV), (dict(ldo=63), INV), (dict(cap=-1), INV), (dict(t=-1), INV), (dict(k=33), INV),
    (dict(cap=(1 << 25) + 1), UNS), (dict(ldx=1 << 33), UNS), (dict(ldo=1 << 33), UNS),
    (dict(x=None), INV), (dict(tr=None), INV), (dict(xs=None), INV), (dict(tr=FAKE + 2), INV), (dict(num=FAKE + 1), INV),
])
def test_dispatch_rows(M, over, status):
    base = dict(x=FAKE, bytes=64, ldx=64, tr=FAKE, t=4, k=2, num=None, cap=8, xs=FAKE, ldo=64)
    refused(M, M.moe_dispatch_rows, base, over, status)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(cap=-1), INV), (dict(d=-1), INV), (dict(ldr=15), INV), (dict(ldy=15), INV), (dict(t=-1), INV),
    (dict(k=0), INV), (dict(cap=(1 << 25) + 1), UNS), (dict(ldr=1 << 33), UNS), (dict(ldy=1 << 33), UNS),
    (dict(rows=None), INV), (dict(tr=None), INV), (dict(y=None), INV), (dict(rows=FAKE + 1), INV), (dict(y=FAKE + 1), INV),
    (dict(w=FAKE + 2), INV), (dict(y=FAKE + 2, dt=1), INV),
])
def test_combine_rows(M, over, status):
    base = dict(rows=FAKE, dt=0, cap=8, d=16, ldr=16, tr=FAKE, w=FAKE, t=4, k=2, y=FAKE, ldy=16)
    refused(M, M.moe_combine_rows, base, over, status)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), INV), (dict(cap=-1), INV), (dict(d=-1), INV), (dict(ldy=15), INV), (dict(ldr=15), INV), (dict(ldd=15), INV),
    (dict(t=(1 << 20) + 1), INV), (dict(k=33), INV), (dict(cap=(1 << 25) + 1), UNS), (dict(ldd=1 << 33), UNS),
    (dict(dy=None), INV), (dict(rows=None), INV), (dict(tr=None), INV), (dict(dy=FAKE + 1), INV), (dict(dr=FAKE + 1), INV),
    (dict(dw=FAKE + 2), INV), (dict(num=FAKE + 2), INV), (dict(w=FAKE + 1), INV),
])
def test_combine_rows_backward(M, over, status):
    base = dict(dy=FAKE, rows=FAKE, dt=0, cap=8, d=16, ldy=16, ldr=16, tr=FAKE, w=FAKE, t=4, k=2, num=None, dr=FAKE, ldd=16,
                dw=FAKE)
    refused(M, M.moe_combine_rows_backward, base, over, status)


def test_row_operators_of_nothing(M):
    M.moe_dispatch_rows(None, 64, 64, None, 0, 2, None, 8, None, 64)
    M.moe_dispatch_rows(None, 0, 0, None, 4, 2, None, 8, None, 0)
    M.moe_combine_rows(None, 0, 8, 16, 16, None, None, 0, 2, None, 16)
    M.moe_combine_rows(None, 0, 8, 0, 0, None, None, 4, 2, None, 0)
    M.moe_combine_rows_backward(None, None, 0, 8, 16, 16, 16, None, None, 4, 2, None, None, 16, None)


def test_no_device_is_a_device_error(M):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(M.MoeError) as ei:
        M.moe_quantize_mx4(FAKE, 0, 4, 64, 64, FAKE, FAKE)
    assert ei.value.status == M.MOE_ERR_DEVICE
    with pytest.raises(M.MoeError) as ei:
        M.moe_sort_tokens(None, 0, 0, 1, 8, FAKE, None, None, None, 0)
    assert ei.value.status == M.MOE_ERR_DEVICE


def test_the_torch_functions_refuse_host_tensors():
    import torch

    from mxfp4_expert_grouped_amd import layer as L
    from mxfp4_expert_grouped_amd import tokens as K
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for call in (lambda: L.quantize_mx4(torch.zeros(4, 64)), lambda: L.dequantize_mx4(z(4, 32), z(4, 2)),
                 lambda: L.linear_mx4(z(4, 32), z(4, 2), z(8, 32), z(8, 2)),
                 lambda: K.sort_tokens(torch.zeros(4, 2, dtype=torch.int32), 3)):
        with pytest.raises(ValueError, match="GPU"):
            call()
