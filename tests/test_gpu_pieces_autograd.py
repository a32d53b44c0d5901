"""The layer's pieces beside torch's own operators on the GPU: what autograd,
views and lazy bits of a tensor ask of a call that goes by addresses."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_expert_grouped_amd import mxmoe
    mxmoe.load_library()
    torch.cuda.set_device(0)
    yield


@pytest.fixture(scope="module")
def L():
    from mxfp4_expert_grouped_amd import layer
    return layer


@pytest.fixture(scope="module")
def K():
    from mxfp4_expert_grouped_amd import tokens
    return tokens


def operands(L, rows, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    return (*L.quantize_mx4(rnd(rows, k)), *L.quantize_mx4(rnd(n, k)))


def test_a_write_to_out_is_seen_by_autograd(L):
    # what another operation saved of the buffer before the product is gone: its gradient is an error, not wrong
    args = operands(L, 5, 8, 64, 1)
    buf = torch.ones(5, 16, device="cuda")
    x = torch.ones(5, 8, device="cuda", requires_grad=True)
    y = x * buf[:, :8]
    version = buf._version
    out = L.linear_mx4(*args, out=buf[:, :8])
    assert buf._version > version and out._version == buf._version
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    # saved after the product it stays, and other calls of the same operands leave it
    y = x * buf[:, :8]
    assert torch.equal(L.linear_mx4(*args, dtype=torch.float32), out)
    y.sum().backward()
    assert torch.equal(x.grad, out)
    # a parameter's values under no_grad, as any operator writes them
    p = torch.nn.Parameter(torch.zeros(5, 8, device="cuda"))
    with torch.no_grad():
        L.linear_mx4(*args, out=p)
    assert torch.equal(p.detach(), out)


def test_a_write_to_an_inference_tensor(L):
    args = operands(L, 5, 8, 64, 2)
    with torch.inference_mode():
        out = torch.zeros(5, 8, device="cuda")
        L.linear_mx4(*args, out=out)
    assert torch.equal(out.clone(), L.linear_mx4(*args, dtype=torch.float32))


def test_an_out_of_one_column(L):
    # the stride along a single column says nothing: a transposed row, a column of a matrix
    args = operands(L, 6, 1, 64, 3)
    ref = L.linear_mx4(*args, dtype=torch.float32)
    out = torch.zeros(1, 6, device="cuda").t()
    assert out.stride() == (1, 6)
    assert torch.equal(L.linear_mx4(*args, out=out), ref)
    wide = torch.zeros(6, 5, device="cuda")
    L.linear_mx4(*args, out=wide.as_strided((6, 1), (5, 3), 2))
    assert torch.equal(wide[:, 2:3], ref) and not wide[:, [0, 1, 3, 4]].any()
    with pytest.raises(ValueError, match="dense rows"):
        L.linear_mx4(*args, out=torch.zeros(1, 1, device="cuda").expand(6, 1))


def lazy(shape, seed):
    """a float32 tensor of which memory holds the negative (the imaginary part of a conjugate), and its values"""
    g = torch.Generator().manual_seed(seed)
    z = torch.complex(torch.randn(shape, generator=g), torch.randn(shape, generator=g)).cuda()
    t = z.conj().imag
    assert t.is_neg()
    return t, -z.imag


@pytest.mark.parametrize("t,d", [(5, 64), (7, 1), (1, 96)])
def test_values_that_memory_does_not_hold(L, K, t, d):
    k, e = 2, 4
    order = K.sort_tokens(torch.randint(0, e, (t, k), generator=torch.Generator().manual_seed(4)).cuda(), e)
    x, xv = lazy((t, d), 5)
    rows, rv = lazy((t * k, d), 6)
    w, wv = lazy((t, k), 7)
    assert torch.equal(K.dispatch(x, order), K.dispatch(xv, order))
    assert torch.equal(K.dispatch_backward(rows, order), K.dispatch_backward(rv, order))
    assert torch.equal(K.combine(rows, w, order), K.combine(rv, wv, order))
    for got, ref in zip(K.combine_backward(x, rows, w, order), K.combine_backward(xv, rv, wv, order)):
        assert torch.equal(got, ref)
    a, b = rows.detach().requires_grad_(), rv.clone().requires_grad_()
    u, v = w.detach().requires_grad_(), wv.clone().requires_grad_()
    for got, ref in zip(torch.autograd.grad(K.combine(a, u, order), (a, u), x), torch.autograd.grad(K.combine(b, v, order), (b, v), xv)):
        assert torch.equal(got, ref)
    # complex elements move as any others do
    z = torch.randn(t, d, dtype=torch.complex64, device="cuda")
    assert torch.equal(K.dispatch(z.conj(), order), K.dispatch(z.conj().resolve_conj(), order))
    if d % 32 == 0:
        for got, ref in zip(L.quantize_mx4(x), L.quantize_mx4(xv)):
            assert torch.equal(got, ref)


def test_an_out_that_memory_does_not_hold_is_refused(L):
    args = operands(L, 4, 8, 64, 8)
    out, _ = lazy((4, 8), 9)
    with pytest.raises(ValueError, match="negated"):
        L.linear_mx4(*args, out=out)
