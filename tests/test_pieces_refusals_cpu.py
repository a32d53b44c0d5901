"""What the torch forms of the layer's pieces refuse before a device is needed."""

import pytest
import torch

from mxfp4_expert_grouped_amd import layer as L


def test_an_out_of_another_type_than_asked_for_is_refused():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    args = (z(4, 32), z(4, 2), z(8, 32), z(8, 2))
    types = (torch.bfloat16, torch.float16, torch.float32)
    for out in types:
        for dtype in (*types, None):
            ok = dtype in (out, None)
            with pytest.raises(ValueError, match="GPU" if ok else "out is"):
                L.linear_mx4(*args, dtype=dtype, out=torch.zeros(4, 8, dtype=out))
