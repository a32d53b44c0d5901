"""The layer's pieces on tensors whose elements and bytes pass 32 bits, looked at
in rows from their start, their middle and their end."""

import numpy as np
import pytest
import torch

from oracle import mx as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_expert_grouped_amd import mxmoe
    mxmoe.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.empty_cache()


def picks(n, each=40):
    return torch.cat([torch.arange(each), torch.arange(n // 2, n // 2 + each), torch.arange(n - each, n)]).cuda()


# 2^31 elements; then more than the 2^31 pieces of 8 that one launch of the conversions takes
@pytest.mark.parametrize("rows", [(1 << 16) + 3, 523775 + 45])
def test_conversions(rows):
    from mxfp4_expert_grouped_amd import layer as L
    cols = 32800
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    block = torch.randn((4097, cols), generator=g, device="cuda").bfloat16()
    for i, part in enumerate(x.split(4097)):
        part.copy_(block[:part.shape[0]])
        part[:, i % cols] = i % 251 + 1  # no two stretches alike
    codes, scales = L.quantize_mx4(x)
    at = picks(rows)
    rc, rs = X.mx_quantize(x[at].cpu().double().numpy(), "e2m1")
    assert np.array_equal(codes[at].cpu().numpy(), rc) and np.array_equal(scales[at].cpu().numpy(), rs)
    del x
    v = L.dequantize_mx4(codes, scales)
    assert np.array_equal(v[at].cpu().double().numpy(), X.mx_decode(rc, rs, "e2m1"))


def test_rows_to_experts_and_back():
    from mxfp4_expert_grouped_amd import tokens as K
    t, k, e, d = (1 << 15) + 1, 8, 96, 8400
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(-1, e, (t, k), generator=g, device="cuda")
    order = K.sort_tokens(ids, e)
    n = int(order.offsets[-1])
    assert n * d > 1 << 31
    x, w, dy = rnd(t, d).bfloat16(), rnd(t, k), rnd(t, d).bfloat16()
    xs = K.dispatch(x, order)
    rows = picks(n)
    token = order.row_src[rows] // k
    assert torch.equal(xs[rows], x[token])
    assert not xs[n:].any()
    tokens = picks(t)
    tr = order.token_row[tokens].long()
    there = (tr >= 0)[:, :, None]
    picked = torch.where(there, xs[tr.clamp(min=0)].double(), 0.0)
    half = torch.finfo(torch.bfloat16).eps / 2
    for weights in (w, None):
        # k products and additions in fp32 (2 k half steps of partial sums), rounded once
        f = weights[tokens].double()[:, :, None] if weights is not None else 1.0
        ref, mag = (picked * f).sum(1), (picked * f).abs().sum(1)
        bound = 2 * k * 2.0 ** -24 * mag
        assert bool(((K.combine(xs, weights, order)[tokens].double() - ref).abs() <= bound + half * (ref.abs() + bound)).all())
    drows, dw = K.combine_backward(dy, xs, w, order)
    ref = dy[token].double() * w.reshape(-1)[order.row_src[rows].long()].double()[:, None]
    assert bool(((drows[rows].double() - ref).abs() <= (2.0 ** -24 + 2 * half) * ref.abs()).all())
    assert not drows[n:].any()
    prod = picked * dy[tokens].double()[:, None, :]
    assert bool(((dw[tokens].double() - prod.sum(2)).abs() <= 2 * d * 2.0 ** -24 * prod.abs().sum(2)).all())
