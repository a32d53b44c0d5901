"""The gated activation far out on the GPU, where its sigmoid is a subnormal
number but its results are not, against float64."""

import pytest
import torch

from test_gpu_experts_kept import X, gpu, near, ref_swiglu, f64  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gates_whose_sigmoid_is_subnormal(X):
    # bf16 has fp32's range, so fp32 tells 88 exp(-88) from zero, and large other factors make it an ordinary number
    g = torch.tensor([-86.5, -87.0, -87.5, -88.0, -88.5, 87.5, 88.0, 88.5]).bfloat16()
    for up, down in ((2.0 ** 100, 2.0 ** 20), (2.0 ** 20, 2.0 ** 100), (-(2.0 ** 60), 2.0 ** 62)):
        h = torch.cat((g, torch.full_like(g, up)))[None]
        da = torch.full_like(g, down)[None]
        # (no more for a sigmoid that comes as zero: it is none here)
        a, dh, _, _ = ref_swiglu(f64(h)[:, :8], f64(h)[:, 8:], f64(da))
        near(X.swiglu(h.cuda()), a, abs(a))
        got, again = X.swiglu_backward(da.cuda(), h.cuda(), need_a=True)
        near(again, a, abs(a))
        near(got, dh, abs(dh))


def test_gates_whose_sigmoid_is_subnormal_from_codes(X):
    # 88 is one of the values that codes have
    h = torch.tensor([[-88.0, -88.0, 2.0 ** 100, -(2.0 ** 100)]]).bfloat16()
    da = torch.tensor([[2.0 ** 10, 2.0 ** 10]]).bfloat16()
    a, dh, _, _ = ref_swiglu(f64(h)[:, :2], f64(h)[:, 2:], f64(da))
    kept_a, kept = X.swiglu_keep(h.cuda())
    assert torch.equal(X.dequantize_mx8(kept[0][:, :2].contiguous(), kept[1][:, :1].contiguous()).cpu(), h[:, :2])
    near(kept_a, a, abs(a))
    got, again = X.swiglu_backward(da.cuda(), kept, need_a=True)
    near(again, a, abs(a))
    near(got, dh, abs(dh))


def test_fp32_gates_whose_sigmoid_is_subnormal(X):
    g = torch.tensor([-87.25, -87.4, -87.9, -88.3, -88.6, -88.7])
    for up, down in ((2.0 ** 100, 2.0 ** 20), (-(2.0 ** 60), 2.0 ** 62)):
        h, da = torch.cat((g, torch.full_like(g, up)))[None], torch.full_like(g, down)[None]
        a, dh, _, _ = ref_swiglu(f64(h)[:, :6], f64(h)[:, 6:], f64(da))
        near(X.swiglu(h.cuda()), a, abs(a))
        near(X.swiglu_backward(da.cuda(), h.cuda())[0], dh, abs(dh))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_gates_below_are_zero(X, dtype):
    g = torch.tensor([-89.0, -95.0, -200.0, -6e4]).to(dtype)
    h = torch.cat((g, torch.full_like(g, 3.0)))[None].cuda()
    assert not X.swiglu(h).any() and not X.swiglu_backward(torch.ones(1, 4, dtype=dtype, device="cuda"), h)[0].any()
