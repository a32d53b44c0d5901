"""Activations in 8 bits and the gated activation on the GPU: codes bit for bit
against the format's oracle, the activation and its gradient against float64."""

import numpy as np
import pytest
import torch

from oracle import mx as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_expert_grouped_amd import mxmoe
    mxmoe.load_library()
    torch.cuda.set_device(0)
    yield


@pytest.fixture(scope="module")
def X():
    from mxfp4_expert_grouped_amd import experts
    return experts


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def ref_codes(v):
    """codes [R, C] and scales of float64 rows of any width; blocks that are not finite: zeros, 255"""
    rows, cols = v.shape
    nb = -(-cols // 32)
    p = np.zeros((rows, nb * 32))
    p[:, :cols] = v
    bad = ~np.isfinite(p.reshape(rows, nb, 32)).all(2)
    p[np.repeat(bad, 32, axis=1)] = 0
    codes, scales = O.mx_quantize(p, "e4m3")
    scales[bad] = 255
    return codes[:, :cols], scales


def ref_values(codes, scales):
    return O.decode_e4m3(np.arange(256))[codes] * np.repeat(O.decode_e8m0(scales), 32, axis=1)[:, :codes.shape[1]]


def matrix(rows, cols, dtype, seed):
    """normal rows of very different size, zeros, subnormal numbers, ties of the grid among them"""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30 if dtype == "bf16" else -12, 8, (rows, 1)))
    v[rng.random((rows, cols)) < 0.05] = 0.0
    ties = rng.random((rows, cols)) < 0.2
    v[ties] = (np.sign(v) * (rng.integers(8, 16, v.shape) + 0.5) / 8)[ties]
    v[rng.random(rows) < 0.1] = 0.0
    v[rng.random(rows) < 0.1] *= 2.0 ** (-100 if dtype != "fp16" else -10)
    return torch.from_numpy(v).to(DT[dtype])


SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (2, 64), (70, 100), (33, 7168), (257, 136), (4, 4099)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_and_values(X, rows, cols, dtype):
    v = matrix(rows, cols, dtype, rows + cols)
    codes, scales = X.quantize_mx8(v.cuda())
    rc, rs = ref_codes(f64(v))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    want = torch.from_numpy(ref_values(rc, rs))
    for out in DT.values():
        assert torch.equal(X.dequantize_mx8(codes, scales, out).cpu(), want.to(out))


def test_codes_of_every_bf16_value(X):
    # a row of 32: the value, a partner that sets the scale, zeros
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for partner in (0.0, 1.0, 2.0 ** -120, 3.0e38):
        v = torch.zeros(1 << 16, 32, dtype=torch.bfloat16)
        v[:, 5] = bits
        v[:, 30] = partner
        codes, scales = X.quantize_mx8(v.cuda())
        rc, rs = ref_codes(f64(v))
        assert np.array_equal(scales.cpu().numpy(), rs)
        assert np.array_equal(codes.cpu().numpy(), rc)


def test_blocks_that_are_not_finite(X):
    v = torch.randn(6, 100)
    v[0, 3], v[1, 40], v[2, 99], v[3, 0], v[3, 64] = float("nan"), float("inf"), -float("inf"), float("nan"), float("inf")
    codes, scales = X.quantize_mx8(v.cuda())
    rc, rs = ref_codes(f64(v))
    assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
    back = X.dequantize_mx8(codes, scales, torch.float32).cpu()
    bad = torch.zeros(6, 100, dtype=torch.bool)
    bad[0, :32] = bad[1, 32:64] = bad[2, 96:] = bad[3, :32] = bad[3, 64:96] = True
    assert torch.equal(back.isnan(), bad)


def test_views_and_nothing(X):
    v = matrix(40, 300, "bf16", 4).cuda()
    for view in (v[::3], v[:, 7:263], v[:, ::2], v.t(), v[:1].expand(5, 300), v[:0], v[:, :0], v[3:4, 1:2]):
        got, want = X.quantize_mx8(view), X.quantize_mx8(view.contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        back = X.dequantize_mx8(*got)
        assert back.shape == view.shape


def ref_swiglu(g, u, da):
    s, t = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    # the magnitudes that errors are relative to.  A sigmoid below 2^-126 (g < -87.3) may come as zero: as a
    # reciprocal it is subnormal, or its exponential infinite.  What that takes from a result is at most
    # 2^-126 times its other factors; near() allows 2^-20 of a magnitude at least, so 2^-106 of them is added.
    m = s + np.where(s < 2.0 ** -126, 2.0 ** -106, 0)
    return g * s * u, np.concatenate([da * u * s * (1 + g * t), da * g * s], axis=1), np.abs(g * m * u), \
        np.concatenate([np.abs(da * u) * m * (1 + np.abs(g) * t), np.abs(da * g) * m], axis=1)


def near(got, ref, mag):
    """Half a step of the result's type; before it, in fp32, an exponential and a reciprocal that are off by
    2^-17 of themselves for 16-bit results, by a few steps for fp32 ones, and ten roundings."""
    step = torch.finfo(got.dtype).eps / 2
    rel = 2.0 ** -20 if got.dtype == torch.float32 else 2.0 ** -15
    tiny = torch.finfo(got.dtype).smallest_normal * step
    g = f64(got)
    assert g.shape == ref.shape
    # (products below the smallest normal fp32 number lose bits on the way)
    err, tol = np.abs(g - ref), step * np.abs(ref) + (1 + step) * rel * mag + tiny + 2.0 ** -120
    assert (err <= tol).all(), f"worst {np.max(err / tol)} of what is allowed"


GLU = [(1, 1), (1, 8), (3, 7), (16, 2048), (5, 31), (40, 33), (129, 136), (70, 1365), (2, 4100)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,f", GLU)
def test_swiglu_and_its_gradient(X, rows, f, dtype):
    gen = torch.Generator().manual_seed(rows * 31 + f)
    h = (torch.randn(rows, 2 * f, generator=gen) * 4).to(DT[dtype])
    da = torch.randn(rows, f, generator=gen).to(DT[dtype])
    h[:, :f][torch.rand(rows, f, generator=gen) < 0.1] *= 20  # far out, where the sigmoid is 0 or 1
    hd = f64(h)
    a, dh, ma, mdh = ref_swiglu(hd[:, :f], hd[:, f:], f64(da))
    hg, dg = h.cuda(), da.cuda()
    near(X.swiglu(hg), a, ma)
    d, again = X.swiglu_backward(dg, hg, need_a=True)
    near(d, dh, mdh)
    near(again, a, ma)
    assert torch.equal(X.swiglu_backward(dg, hg)[0], d) and X.swiglu_backward(dg, hg)[1] is None
    # in 8 bits: the codes of both halves, and the formulas at their values
    kept_a, (codes, scales) = X.swiglu_keep(hg)
    assert torch.equal(kept_a, X.swiglu(hg))
    (cg, sg), (cu, su) = ref_codes(hd[:, :f]), ref_codes(hd[:, f:])
    assert np.array_equal(codes.cpu().numpy(), np.concatenate([cg, cu], axis=1))
    assert np.array_equal(scales.cpu().numpy(), np.concatenate([sg, su], axis=1))
    a, dh, ma, mdh = ref_swiglu(ref_values(cg, sg), ref_values(cu, su), f64(da))
    d, again = X.swiglu_backward(dg, (codes, scales), need_a=True)
    near(d, dh, mdh)
    near(again, a, ma)
    # through autograd
    for checkpoint, want in ((None, X.swiglu_backward(dg, hg)[0]), ("mx8", d)):
        leaf = hg.clone().requires_grad_()
        out = X.swiglu(leaf, checkpoint=checkpoint)
        assert torch.equal(out, kept_a)
        assert torch.equal(torch.autograd.grad(out, leaf, dg)[0], want)


def test_swiglu_gradient_against_differences(X):
    gen = torch.Generator().manual_seed(3)
    h, da = torch.randn(4, 22, generator=gen).cuda(), torch.randn(4, 11, generator=gen).cuda()
    dh = X.swiglu_backward(da, h)[0].double()
    step = 2.0 ** -7
    for c in range(22):
        e = torch.zeros_like(h)
        e[:, c] = step
        slope = ((X.swiglu(h + e).double() - X.swiglu(h - e).double()) * da.double()).sum(1) / (2 * step)
        # the third derivative times step^2 / 6, and roundings of a (of size up to 2^4) over the step
        assert ((slope - dh[:, c]).abs() <= 2.0 ** -14 * 16 + 2.0 ** -24 * 2 ** 4 * 64 * 11).all()


def test_swiglu_values_that_are_not_finite(X):
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([inf, nan, 1.0, 1.0, 100.0, -200.0, 3.0e38, -3.0e38])
    u = torch.tensor([1.0, 1.0, inf, nan, 2.0, 2.0, 1.0, 1.0])
    a = X.swiglu(torch.cat((g, u))[None].cuda()).cpu()[0]
    assert a[0] == inf and a[1].isnan() and a[2] == inf and a[3].isnan() and a[4] == 200.0 and a[5] == 0 and a[6] == g[6] and a[7] == 0
    dh = X.swiglu_backward(torch.ones(1, 8).cuda(), torch.cat((g, u))[None].cuda())[0].cpu()[0]
    assert (dh[4], dh[5], dh[12], dh[13]) == (2.0, 0.0, 100.0, 0.0) and dh[6] == 1.0 and dh[7] == 0
    assert dh[1].isnan() and dh[3].isnan()


def test_swiglu_views_and_nothing(X):
    h, da = torch.randn(50, 200).bfloat16().cuda(), torch.randn(50, 50).bfloat16().cuda()
    for view, d in ((h[::2, :100], da[::2]), (h[:, 3:103], da), (h[:, ::2], da), (h[:0, :100], da[:0]), (h[:, :0], da[:, :0]), (h[:1, :100].expand(9, 100), da[:1].expand(9, 50))):
        assert torch.equal(X.swiglu(view), X.swiglu(view.contiguous()))
        assert torch.equal(X.swiglu_backward(d, view)[0], X.swiglu_backward(d.contiguous(), view.contiguous())[0])
        kept = X.swiglu_keep(view)[1]
        assert torch.equal(X.swiglu_backward(d, kept)[0], X.swiglu_backward(d.contiguous(), kept)[0])
