"""That the check of the gradients at kept values tells the forms of their
operands apart: a mistake in one of them, planted here in the formulas, does
not pass."""

import numpy as np
import pytest
import torch

import test_gpu_experts_kept_gradients as G


@pytest.mark.parametrize("dtype,rows,experts,d,f", G.SIZES)
def test_mistakes_do_not_pass(dtype, rows, experts, d, f):
    *tensors, cuts = G.inputs(dtype, rows, experts, d, f)
    x, gu, dn, dy = (t.double().numpy() for t in tensors)
    h = np.concatenate([x[a:b] @ gu[e].T for e, (a, b) in enumerate(zip(cuts, cuts[1:]))])
    h = torch.from_numpy(h).to(G.DT[dtype]).double().numpy()
    xk, hk, joined = G.kept(x, dtype, False), G.kept(h, dtype, True), G.kept(h, dtype, False)
    right = dict(dw_x=xk, act_h=hk, again_h=hk)
    ranges = G.gradients(x, gu, dn, dy, h, cuts, dtype, **right)
    assert all(G.inside(r[0], r) for r in ranges)
    plain = G.gradients(x, gu, dn, dy, h, cuts, dtype, x, h, h)
    # one operand in another form each, and the gradients that it enters
    for wrong, enters in ((dict(dw_x=x), (1,)), (dict(act_h=h), (0, 1)), (dict(again_h=h), (2,)), (dict(dw_x=G.kept(x * 1.03, dtype, False)), (1,)),
                          (dict(act_h=np.roll(hk, 1, axis=0)), (0, 1)), (dict(again_h=np.roll(hk, f, axis=1)), (2,))):
        got = G.gradients(x, gu, dn, dy, h, cuts, dtype, **{**right, **wrong})
        for n in range(3):
            assert G.inside(got[n][0], ranges[n]) == (n not in enters), (list(wrong), n)
    # gate and up have blocks of their own: where a block reaches over both, it shows
    if f % 32:
        got = G.gradients(x, gu, dn, dy, h, cuts, dtype, xk, joined, joined)
        assert not G.inside(got[0][0], ranges[0]) and not G.inside(got[2][0], ranges[2])
    # and the other way round, rows kept as they are
    for n in range(3):
        assert not G.inside(ranges[n][0], plain[n])
