"""16-bit products of rows sorted by expert and their gradients on the GPU,
against float64.

How far a result may be off: its rounding, half a step of its type, and the
fp32 sum, whose error for L products is at most about L u times the sum of
their magnitudes; u is taken as 2^-23, a whole step, since how the matrix
cores round inside a sum is not documented.
"""

import numpy as np
import pytest
import torch

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


def near(got, ref, mag, length):
    """got (rounded to its type) against ref, a sum of `length` products whose magnitudes sum to mag (float64)"""
    assert got.shape == ref.shape
    step = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * step  # half a step of the subnormal numbers
    err = (got.double() - ref).abs()
    tol = step * ref.abs() + tiny + (1 + step) * length * 2.0 ** -23 * mag
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst by {float((err / tol.clamp(min=1e-300)).max()):.3g} of what is allowed, first at {bad.nonzero()[0].tolist()}"


def ragged(rows, mats, kind, seed):
    """offsets [mats + 1] as a list"""
    rng = np.random.default_rng(seed)
    if kind == "even":
        cuts = np.linspace(0, rows, mats + 1).round()
    elif kind == "ragged":     # matrices without rows among them, all rows covered
        cuts = np.sort(rng.integers(0, rows + 1, mats + 1))
        cuts[0], cuts[-1] = 0, rows
    elif kind == "uncovered":  # rows of no matrix in front and behind
        cuts = np.sort(rng.integers(rows // 5, rows - rows // 4 + 1, mats + 1))
    elif kind == "one":        # everything to one in the middle
        cuts = np.where(np.arange(mats + 1) > mats // 2, rows, 0)
    elif kind == "none":
        cuts = np.full(mats + 1, rows // 2)
    return [int(c) for c in cuts]


def data(rows, mats, n, k, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    return rnd(rows, k), rnd(max(mats, 1), n, k), rnd(rows, n)


def dx_of(X, dy, w, off=None):
    dx, none = X.linear_backward(dy, None, w, off, need_w=False)
    assert none is None
    return dx


def dw_of(X, dy, x, off=None, dtype=None):
    none, dw = X.linear_backward(dy, x, None, off, need_x=False, w_dtype=dtype)
    assert none is None
    return dw


def check_all(X, x, w, dy, offsets, dw_dtype=None):
    """the product and both gradients by the functions without autograd"""
    rows, (mats, n, k) = x.shape[0], w.shape
    grouped = offsets is not None
    cuts = offsets if grouped else [0, rows]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda") if grouped else None
    we = w if grouped else w[0]
    y, (dx, dw) = X.linear(x, we, off), X.linear_backward(dy, x, we, off, w_dtype=dw_dtype)
    assert torch.equal(dx, dx_of(X, dy, we, off)) and torch.equal(dw, dw_of(X, dy, x, off, dw_dtype))
    zero = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")  # noqa: E731
    ry, my, rdx, mdx, rdw, mdw = zero(rows, n), zero(rows, n), zero(rows, k), zero(rows, k), zero(mats, n, k), zero(mats, n, k)
    for e in range(mats):
        s = slice(cuts[e], cuts[e + 1])
        xe, ye, wd = x[s].double(), dy[s].double(), w[e].double()
        ry[s], my[s] = xe @ wd.T, xe.abs() @ wd.abs().T
        rdx[s], mdx[s] = ye @ wd, ye.abs() @ wd.abs()
        rdw[e], mdw[e] = ye.T @ xe, ye.abs().T @ xe.abs()
    near(y, ry, my, k)
    near(dx, rdx, mdx, n)
    near(dw, rdw if grouped else rdw[0], mdw if grouped else mdw[0], max(b - a for a, b in zip(cuts, cuts[1:])))
    return y, dx, dw


# rows, matrices (0: one without offsets), n, k
SIZES = [(1, 0, 1, 1), (1, 0, 8, 8), (3, 0, 64, 64), (64, 0, 256, 64), (65, 0, 257, 65), (300, 0, 512, 320), (1000, 0, 24, 4096),
         (257, 1, 256, 256), (40, 3, 72, 136), (500, 7, 264, 200), (999, 13, 131, 77), (2000, 40, 520, 72), (128, 300, 32, 40),
         (5000, 3, 128, 128), (700, 2, 1000, 1032), (77, 5, 2, 3), (4096, 9, 384, 640),
         # with those above, every kernel and several tiles for a workgroup (asked of the rule on the CPU)
         (583, 40, 5593, 40), (1543, 17, 4598, 39), (22940, 0, 1336, 34), (3161, 40, 76, 3296), (1463, 17, 72, 7248),
         (32685, 40, 94, 36), (8598, 40, 2408, 32), (21, 17, 32, 7776), (9063, 2, 40, 2584)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,mats,n,k", SIZES)
def test_products_and_gradients(X, rows, mats, n, k, dtype):
    x, w, dy = data(rows, mats, n, k, dtype, rows + n)
    if not mats:
        check_all(X, x, w, dy, None)
        check_all(X, x, w, dy, None, torch.float32)
        return
    for kind in ("even", "ragged", "uncovered", "one", "none"):
        check_all(X, x, w, dy, ragged(rows, mats, kind, k), torch.float32 if kind == "even" else None)


@pytest.mark.parametrize("rows,mats,n,k,dtype", [(300, 5, 136, 256, "bf16"), (513, 0, 72, 100, "bf16"), (90, 4, 33, 31, "fp16"), (1, 1, 8, 5, "bf16"),
                                                 (0, 3, 16, 40, "bf16")])
def test_weights_gradient_from_rows_in_8_bits(X, rows, mats, n, k, dtype):
    x, w, dy = data(rows, mats, n, k, dtype, 7)
    kept = X.quantize_mx8(x)
    values = X.dequantize_mx8(*kept, DT[dtype])
    off = torch.tensor(ragged(rows, mats, "uncovered", 1), dtype=torch.int32, device="cuda") if mats else None
    for out in (None, torch.float32):
        assert torch.equal(dw_of(X, dy, kept, off, out), dw_of(X, dy, values, off, out))


def test_rows_with_a_nan_scale_reach_their_columns_only(X):
    x, _, dy = data(40, 2, 16, 70, "bf16", 9)
    x[3, 33] = float("inf")  # in the first matrix
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    dw = dw_of(X, dy, X.quantize_mx8(x), off)
    assert dw[0, :, 32:64].isnan().all() and not dw[0, :, :32].isnan().any() and not dw[0, :, 64:].isnan().any() and not dw[1].isnan().any()


def test_rows_of_no_matrix_are_not_read(X):
    # what lies there, NaN included, reaches nothing
    x, w, dy = data(200, 3, 64, 72, "bf16", 2)
    off = torch.tensor([30, 90, 90, 150], dtype=torch.int32, device="cuda")
    want = X.linear(x, w, off), dx_of(X, dy, w, off), dw_of(X, dy, x, off)
    for t in (x, dy):
        t[:30], t[150:] = float("nan"), float("inf")
    got = X.linear(x, w, off), dx_of(X, dy, w, off), dw_of(X, dy, x, off)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not want[0][:30].any() and not want[0][150:].any() and not want[1][:30].any() and not want[2][1].any()


def test_views(X):
    x, w, dy = data(120, 3, 128, 96, "bf16", 5)
    off = torch.tensor([0, 50, 70, 120], dtype=torch.int32, device="cuda")
    want = X.linear(x, w, off), dx_of(X, dy, w, off), dw_of(X, dy, x, off)
    big = lambda t, left, right: torch.nn.functional.pad(t, (left, right), value=float("nan"))[:, left:left + t.shape[1]]  # noqa: E731
    for xv, wv, dv, ov in ((big(x, 8, 8), w, big(dy, 0, 8), off), (big(x, 3, 2), w, big(dy, 1, 1), off),
                           (x.t().contiguous().t(), w.transpose(1, 2).contiguous().transpose(1, 2), dy.t().contiguous().t(), off),
                           (x, w, dy, torch.stack((off, off), 1)[:, 0]), (x.repeat_interleave(2, 0)[::2], w, dy.repeat_interleave(2, 0)[1::2], off)):
        got = X.linear(xv, wv, ov), dx_of(X, dv, wv, ov), dw_of(X, dv, xv, ov)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_broadcast_gradient(X):
    x, w, _ = data(33, 0, 40, 56, "bf16", 6)
    xl, wl = x.requires_grad_(), w[0].requires_grad_()
    gx, gw = torch.autograd.grad(X.linear(xl, wl).sum(), (xl, wl))
    one = torch.ones(33, 40, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(gx, dx_of(X, one, wl.detach())) and torch.equal(gw, dw_of(X, one, xl.detach()))


def test_sizes_of_zero(X):
    e = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert X.linear(e(0, 8), e(5, 8)).shape == (0, 5)
    assert X.linear(e(4, 8), e(0, 8)).shape == (4, 0)
    assert torch.equal(X.linear(e(4, 0), e(5, 0)), e(4, 5) * 0)
    assert torch.equal(X.linear(e(4, 8), e(3, 5, 8), off), e(4, 5) * 0)
    assert torch.equal(dx_of(X, e(4, 0), e(0, 8)), e(4, 8) * 0)
    for x in (e(0, 8), X.quantize_mx8(e(0, 8))):
        assert torch.equal(dw_of(X, e(0, 5), x), e(5, 8) * 0)
        assert torch.equal(dw_of(X, e(0, 5), x, off), e(3, 5, 8) * 0)
    assert dw_of(X, e(3, 0), e(3, 8)).shape == (0, 8) and dw_of(X, e(3, 5), e(3, 0)).shape == (5, 0)


def test_offsets_out_of_range_stay_inside(X):
    # values that no sort gives: taken as the nearer end, never outside a buffer
    x, w, dy = data(50, 3, 24, 32, "bf16", 8)
    wild = torch.tensor([-7, 10, 1 << 30, -5], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 10, 50, 50], dtype=torch.int32, device="cuda")
    y, t = X.linear(x, w, wild), X.linear(x, w, tame)
    assert torch.equal(y, t)
    assert torch.equal(dw_of(X, dy, x, wild)[:2], dw_of(X, dy, x, tame)[:2])
