"""How many roundings a product passes through in the gradient of the routing
weights, and orders of many chunks of pairs."""

import math

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
def K():
    from mxfp4_expert_grouped_amd import tokens
    return tokens


def one_row_each(K, t):
    """the order of t tokens with one choice each, token i's row being row i"""
    return K.sort_tokens(torch.zeros(t, 1, dtype=torch.int32, device="cuda"), 1)


def roundings(d, dtype):
    # 64 lanes with a sum for each element of a 16-byte piece: a multiply-add rounds once for each of a lane's
    # pieces, then the sums of a piece are joined in pairs and those of the lanes
    vec = 16 // DT[dtype].itemsize
    return math.ceil(math.ceil(d / vec) / 64) + int(math.log2(vec)) + 6


def dw_of(K, dy, rows, dtype):
    order = one_row_each(K, dy.shape[0])
    _, dw = K.combine_backward(dy.to(DT[dtype]).cuda(), rows.to(DT[dtype]).cuda(), None, order)
    return dw.cpu().double()[:, 0]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [7168, 7165, 4096, 1000])
def test_weight_gradients_lose_no_more_than_their_roundings(K, d, dtype):
    # token i: a product of 1 first in lane i's share, and products just below half of 1's last place everywhere
    # else in it: each vanishes that is added to the 1, and none that is added elsewhere
    vec = 16 // DT[dtype].itemsize
    lane = (torch.arange(d) // vec) % 64
    mine = lane[None, :] == torch.arange(64)[:, None]
    rows = torch.where(mine, 2.0 ** -12 * 255 / 256, 0.0).double()
    dy = torch.full((64, d), 2.0 ** -12, dtype=torch.float64)
    first = torch.arange(64) * vec
    rows[torch.arange(64), first] = 1.0
    dy[torch.arange(64), first] = 1.0
    ref = (rows * dy).sum(1)  # exact: every product is a multiple of 2^-32, and the sum is below 2
    # (all positive: the sum is the sum of magnitudes; one rounding more covers the second order)
    assert ((dw_of(K, dy, rows, dtype) - ref).abs() <= (roundings(d, dtype) + 1) * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [1, 5, 64, 513, 7168])
def test_weight_gradients_of_random_rows(K, d, dtype):
    g = torch.Generator().manual_seed(d)
    dy, rows = (torch.randn(130, d, generator=g).to(DT[dtype]).double() for _ in range(2))
    ref, mag = (dy * rows).sum(1), (dy * rows).abs().sum(1)
    assert ((dw_of(K, dy, rows, dtype) - ref).abs() <= (roundings(d, dtype) + 1) * 2.0 ** -24 * mag).all()


# pairs in chunks of 2048 up to 2^20 pairs (128 chunks: the last number that every workgroup sums itself; 129 and
# more: a launch of their own sums them), of 4096 above: 257 to the documented limits' 8192
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("t,k,e", [(131072, 2, 896), (131071, 2, 1024), (131073, 2, 1024), (262145, 1, 17), (100001, 5, 300),
                                   (32768, 16, 896), (262144, 4, 1000), (1048576, 1, 1), (65537, 16, 896), (1048575, 3, 77)])
def test_orders_of_many_chunks(K, t, k, e, dtype):
    check_order(K, t, k, e, dtype)


def test_the_order_of_the_most_pairs(K):
    check_order(K, 1 << 20, 32, 1024, torch.int32)


def check_order(K, t, k, e, dtype):
    # experts of very different size, a sixth of the choices dropped, whole stretches of them too
    rng = np.random.default_rng(t + k + e)
    ids = np.minimum(rng.integers(0, e, (t, k)), rng.integers(0, e + e // 5 + 1, (t, k))).astype(np.int16)
    ids[rng.random((t, k)) < 1 / 6] = -1
    ids[t // 3:t // 3 + 3000] = e
    flat = ids.reshape(-1)
    kept = np.flatnonzero((flat >= 0) & (flat < e))
    src = kept[np.argsort(flat[kept], kind="stable")]
    order = K.sort_tokens(torch.from_numpy(ids).to(dtype).cuda(), e)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=e))])
    assert np.array_equal(order.offsets.cpu().numpy(), offsets)
    row_src = order.row_src.cpu().numpy()
    assert np.array_equal(row_src[:src.size], src) and (row_src[src.size:] == -1).all()
    token_row = np.full(flat.size, -1, dtype=np.int32)
    token_row[src] = np.arange(src.size, dtype=np.int32)
    assert np.array_equal(order.token_row.cpu().numpy().reshape(-1), token_row)
