"""What the torch forms of the layer's pieces refuse before a device is needed."""

import copy
import pickle

import pytest
import torch

from mxfp4_expert_grouped_amd import layer as L
from mxfp4_expert_grouped_amd import tokens as K


def test_an_out_of_another_type_than_asked_for_is_refused():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    args = (z(4, 32), z(4, 2), z(8, 32), z(8, 2))
    types = (torch.bfloat16, torch.float16, torch.float32)
    for out in types:
        for dtype in (*types, None):
            ok = dtype in (out, None)
            with pytest.raises(ValueError, match="GPU" if ok else "out is"):
                L.linear_mx4(*args, dtype=dtype, out=torch.zeros(4, 8, dtype=out))


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("name,bad", [
    ("offsets", ints(5).long()), ("offsets", ints(1, 5)), ("offsets", ints(1)), ("offsets", ints(10)[::2]),
    ("offsets", ints(1).expand(5)), ("offsets", torch.zeros(5)), ("offsets", torch.empty(5, dtype=torch.int32, device="meta")),
    ("row_src", ints(8).long()), ("row_src", ints(7)), ("row_src", ints(4, 2)), ("row_src", ints(16)[::2]),
    ("token_row", ints(4, 2).long()), ("token_row", ints(8)), ("token_row", ints(2, 4).t()), ("token_row", ints(1, 2).expand(4, 2)),
    ("token_row", ints(8, 2)[::2]), ("token_row", ints(5, 2)), ("token_row", torch.empty((4, 2), dtype=torch.int32, device="meta")),
])
def test_an_order_of_tensors_that_cannot_be_one_is_refused(name, bad):
    # the kernels read these by address: one short, strided, of another type or device would be read past its end
    good = dict(offsets=ints(5), row_src=ints(8), token_row=ints(4, 2))
    K.TokenOrder(**good)
    with pytest.raises(ValueError):
        K.TokenOrder(**{**good, name: bad})


def test_an_order_does_not_change():
    order = K.TokenOrder(ints(5), ints(8), ints(4, 2))
    assert (order.num_experts, order.num_tokens, order.top_k, order.capacity) == (4, 4, 2, 8)
    for name in ("offsets", "row_src", "token_row", "other"):
        with pytest.raises(AttributeError):
            setattr(order, name, ints(3))
    for again in (copy.copy(order), copy.deepcopy(order), pickle.loads(pickle.dumps(order))):
        assert all(torch.equal(getattr(again, n), getattr(order, n)) for n in K.TokenOrder.__slots__)
    assert K.TokenOrder(ints(5), ints(0), ints(0, 2)).capacity == 0


def test_a_product_of_more_tiles_than_a_launch_counts_is_refused():
    # (its y would be larger than any memory; the tiles past the limit would have been left out)
    from mxfp4_expert_grouped_amd import mxmoe as M
    fake = 1 << 20  # never dereferenced: there is no such device, or the call fails its checks

    def status(rows, mats, n):
        with pytest.raises(M.MoeError) as ei:
            M.moe_linear_mx4(fake, fake, rows, fake, fake, mats, fake, n, 128, fake, M.MOE_SRC_BF16, n)
        return ei.value.status

    for rows, mats, n in ((1 << 25, 1, 1 << 20), (1 << 24, 1, 1 << 20), (1 << 25, 1024, 1 << 19), (64 * ((1 << 18) - 1), 2, 1 << 20)):
        assert status(rows, mats, n) == M.MOE_ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        for rows, mats, n in ((64 * ((1 << 18) - 1), 1, 1 << 20), (1 << 25, 64, 1 << 18)):
            assert status(rows, mats, n) == M.MOE_ERR_DEVICE
