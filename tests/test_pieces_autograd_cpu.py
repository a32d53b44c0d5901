"""What the layer's pieces owe to autograd, as far as it is settled before a
device is needed: what they cannot differentiate is refused, not dropped."""

import pytest
import torch
from torch.autograd import forward_ad

from mxfp4_expert_grouped_amd import layer as L
from mxfp4_expert_grouped_amd import tokens as K


def order(t, k, e):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return K.TokenOrder(i32(e + 1), i32(t * k), i32(t, k))


TANGENT_CALLS = {
    "dispatch": lambda d, o: K.dispatch(d(4, 8), o),
    "combine_rows": lambda d, o: K.combine(d(8, 8), None, o),
    "combine_weights": lambda d, o: K.combine(torch.zeros(8, 8), d(4, 2), o),
    "dispatch_backward": lambda d, o: K.dispatch_backward(d(8, 8), o),
    "combine_backward_dy": lambda d, o: K.combine_backward(d(4, 8), torch.zeros(8, 8), None, o),
    "combine_backward_rows": lambda d, o: K.combine_backward(torch.zeros(4, 8), d(8, 8), None, o),
    "combine_backward_weights": lambda d, o: K.combine_backward(torch.zeros(4, 8), torch.zeros(8, 8), d(4, 2), o),
    "quantize_mx4": lambda d, o: L.quantize_mx4(d(4, 32)),
    "linear_mx4_out": lambda d, o: L.linear_mx4(*[torch.zeros(s, dtype=torch.uint8) for s in ((4, 32), (4, 2), (8, 32), (8, 2))],
                                                out=d(4, 8)),
}


@pytest.mark.parametrize("call", list(TANGENT_CALLS))
def test_a_forward_mode_tangent_is_refused(call):
    # (make_dual's tensors do not require a gradient and have their values' address)
    with forward_ad.dual_level():
        dual = lambda *s: forward_ad.make_dual(torch.ones(s), torch.ones(s))  # noqa: E731
        with pytest.raises(NotImplementedError, match="tangent"):
            TANGENT_CALLS[call](dual, order(4, 2, 3))
        with pytest.raises(ValueError, match="GPU"):  # tensors without one go on to the other checks
            TANGENT_CALLS[call](lambda *s: torch.ones(s), order(4, 2, 3))


def test_an_out_that_requires_a_gradient_is_refused():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    args = (z(4, 32), z(4, 2), z(8, 32), z(8, 2))
    leaf = torch.zeros(4, 8, requires_grad=True)
    for out in (leaf, leaf * 2, leaf[:]):
        with pytest.raises(ValueError, match="gradient"):
            L.linear_mx4(*args, out=out)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # as for any write into it: on to the other checks
            L.linear_mx4(*args, out=out)


def test_quantising_what_requires_a_gradient_is_refused():
    # the codes could not pass it on: a chain through them would train without a word
    leaf = torch.zeros(4, 32, requires_grad=True)
    for src in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            L.quantize_mx4(src)
        for call in (lambda: L.quantize_mx4(src.detach()), torch.no_grad()(lambda: L.quantize_mx4(src))):
            with pytest.raises(ValueError, match="GPU"):  # on to the other checks
                call()
