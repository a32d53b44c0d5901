"""16-bit products of rows sorted by expert on operands whose sums are exact, on
the GPU: whole numbers from -2 to 2, of which every partial sum stays below
2^24, so that fp32 holds it whatever the order.  A result is then the sum,
rounded once to its type, and compared for equality: one product too many or
too few in a sum of any length shows.
"""

import numpy as np
import pytest
import torch

from test_gpu_experts import DT, X, gpu, ragged  # noqa: F401

pytestmark = pytest.mark.gpu

# rows, matrices (0: one without offsets), n, k: for each pass, height of a tile and way of storing a workgroup
# with several tiles, in sums of several steps; and last rounds of tiles that two workgroups share (asked of the
# rule on the CPU)
SIZES = [(31254, 20, 113, 322), (5429, 40, 49, 1976), (30798, 20, 24, 328), (36297, 0, 258, 263), (5355, 20, 40, 4880),
         (32875, 40, 264, 288), (15625, 20, 31, 784), (1368, 20, 258, 1400), (15662, 20, 48, 424), (31257, 20, 400, 52),
         (2636, 20, 2128, 24), (30813, 20, 656, 64), (5210, 20, 4987, 27), (125, 40, 256, 1557), (2604, 40, 1293, 24),
         (15574, 20, 544, 56), (5608, 20, 24, 3109), (10329, 40, 24, 1856), (6291, 20, 3255, 26), (5130, 20, 3552, 32),
         (282, 20, 4427, 24), (118, 40, 24, 1631), (108, 40, 1670, 27), (22940, 0, 1336, 34), (30000, 0, 128, 256)]
KINDS = ("even", "ragged", "uncovered")


def cuts_of(rows, mats, kind, k):
    return ragged(rows, mats, kind, k) if mats else [0, rows]


def whole(shape, seed):
    """whole numbers from -2 to 2, few of them zero, as float64 on the CPU"""
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.choice(np.array([-2, -1, -1, 0, 1, 1, 2], dtype=np.float64), shape))


def operands(rows, mats, n, k):
    return whole((rows, k), rows), whole((max(1, mats), n, k), n), whole((rows, n), k)


def sums(x, w, dy, cuts):
    """y, dx, dw in float64"""
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w)
    for e in range(w.shape[0]):
        s = slice(cuts[e], cuts[e + 1])
        y[s], dx[s], dw[e] = x[s] @ w[e].T, dy[s] @ w[e], dy[s].T @ x[s]
    return y, dx, dw


def equal(got, want):
    assert got.shape == want.shape
    bad = got != want.to(got.dtype)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,mats,n,k", SIZES)
def test_sums_are_exact(X, rows, mats, n, k, dtype):
    x, w, dy = (t.cuda() for t in operands(rows, mats, n, k))
    x16, w16, dy16 = (t.to(DT[dtype]) for t in (x, w, dy))
    for kind in KINDS if mats else KINDS[:1]:
        cuts = cuts_of(rows, mats, kind, k)
        off = torch.tensor(cuts, dtype=torch.int32, device="cuda") if mats else None
        we = w16 if mats else w16[0]
        y, dx, dw = sums(x, w, dy, cuts)
        xs, dys = x16.clone(), dy16.clone()
        for t in (xs, dys):  # what no matrix has reaches nothing
            t[:cuts[0]], t[cuts[-1]:] = float("nan"), float("inf")
        equal(X.linear(xs, we, off), y)
        for w_dtype in (None, torch.float32):
            got_dx, got_dw = X.linear_backward(dys, xs, we, off, w_dtype=w_dtype)
            equal(got_dx, dx)
            equal(got_dw, dw if mats else dw[0])


def test_sums_past_32_bits_are_exact(X):
    # x of 5 GB, dy and y of 4.7 GB, dx of 5 GB; sums of 300000 rows
    rows, n, k = 600011, 3904, 4160
    g = torch.Generator(device="cuda").manual_seed(1)

    def few(*shape):  # -1, 0 and 1
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for part in t.split(1 << 15):
            part.copy_(torch.randint(-1, 2, part.shape, generator=g, device="cuda", dtype=torch.int8))
        return t

    x, w, dy = few(rows, k), few(2, n, k), few(rows, n)
    cuts = [5, 299999, rows]
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    y = X.linear(x, w, off)
    dx, dw = X.linear_backward(dy, x, w, off)
    none, dw32 = X.linear_backward(dy, x, None, off, need_x=False, w_dtype=torch.float32)
    assert none is None and not y[:5].any() and not dx[:5].any()
    for e in range(2):
        want = torch.zeros(n, k, device="cuda")
        we = w[e].float()
        for a in range(cuts[e], cuts[e + 1], 1 << 15):
            s = slice(a, min(a + (1 << 15), cuts[e + 1]))
            xs, dys = x[s].float(), dy[s].float()
            equal(y[s], xs @ we.T)
            equal(dx[s], dys @ we)
            want += dys.T @ xs
        equal(dw32[e], want)
        equal(dw[e], want)
