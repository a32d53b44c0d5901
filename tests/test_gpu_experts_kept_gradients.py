"""Gradients of the experts' network at rows kept in 8 bits, on the GPU, against
the formulas in float64 at the values that the format's oracle keeps: which
operand enters which gradient in which form, and nothing looser than the
roundings to 16 bits.

What is computed is rounded once where the operators' documentation says so,
and carried on as the rounded value with a range: a rounding whose argument may
lie on either side of a border gives two values, all others one.
"""

import numpy as np
import pytest
import torch

from test_gpu_experts_kept import X, f64, gpu, ref_codes, ref_values  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
STEP = 2.0 ** -23  # of an fp32 sum, for each of its products
ACTIVATION = 2.0 ** -15  # of an activation's factors before their rounding, relative

# dtype, rows, experts, d, d_ff
SIZES = [("bf16", 64, 3, 96, 32), ("fp16", 40, 2, 64, 48), ("bf16", 300, 5, 72, 33), ("fp16", 90, 1, 31, 20)]


def rounded(v, err, dt):
    """(value, range) of v, known to within err, rounded to dt"""
    to = lambda a: torch.from_numpy(a).to(DT[dt]).double().numpy()  # noqa: E731
    r = to(v)
    return r, np.maximum(np.abs(to(v + err) - r), np.abs(to(v - err) - r))


def product(a, b, dt):
    """a @ b of (value, range) pairs, rounded"""
    (av, ar), (bv, br) = a, b
    top = (np.abs(av) + ar) @ (np.abs(bv) + br)
    return rounded(av @ bv, top - np.abs(av) @ np.abs(bv) + av.shape[1] * STEP * top, dt)


def kept(v, dt, halves):
    """the values that stand for v in 8 bits, in dt"""
    parts = np.split(v, 2, axis=1) if halves else [v]
    values = np.concatenate([ref_values(*ref_codes(p)) for p in parts], axis=1)
    return values if halves else torch.from_numpy(values).to(DT[dt]).double().numpy()


def gradients(x, gu, dn, dy, h, cuts, dt, dw_x, act_h, again_h):
    """(value, range) of dx, dw_gate_up, dw_down of one network: dw_x the rows of dw_gate_up, act_h the input at
    which the activation's gradient is taken, again_h that of the activation in dw_down"""
    f = dn.shape[2]
    out = [(np.zeros(s), np.zeros(s)) for s in (x.shape, gu.shape, dn.shape)]
    exact = lambda v: (v, np.zeros_like(v))  # noqa: E731

    def put(n, at, pair):
        out[n][0][at], out[n][1][at] = pair

    for e in range(len(gu)):
        s = slice(cuts[e], cuts[e + 1])
        da, rda = product(exact(dy[s]), exact(dn[e]), dt)
        g, u = act_h[s, :f], act_h[s, f:]
        p = 1 / (1 + np.exp(-g))
        by_g, by_u = u * p * (1 + g * (1 - p)), g * p
        most_g = np.abs(u) * p * (1 + np.abs(g) * (1 - p))
        v = np.concatenate([da * by_g, da * by_u], axis=1)
        err = np.concatenate([rda * np.abs(by_g) + ACTIVATION * (np.abs(da) + rda) * most_g,
                              (rda + ACTIVATION * (np.abs(da) + rda)) * np.abs(by_u)], axis=1)
        dh = rounded(v, err, dt)
        ga, ua = again_h[s, :f], again_h[s, f:]
        a = ga / (1 + np.exp(-ga)) * ua
        a = rounded(a, ACTIVATION * np.abs(a), dt)
        put(0, s, product(dh, exact(gu[e]), dt))
        put(1, e, product((dh[0].T, dh[1].T), exact(dw_x[s]), dt))
        put(2, e, product(exact(dy[s].T.copy()), a, dt))
    return out


def inside(got, pair):
    """whether got (float64, values of the type) is in a range"""
    value, within = pair
    return bool((np.abs(got - value) <= within).all())


def inputs(dt, rows, experts, d, f):
    rng = np.random.default_rng(rows + d)
    to = lambda v: torch.from_numpy(v).to(DT[dt])  # noqa: E731
    x = to(rng.standard_normal((rows, d)) * np.exp(rng.standard_normal((rows, 1)) / 2))
    gu, dn = to(rng.standard_normal((experts, 2 * f, d)) * d ** -0.5), to(rng.standard_normal((experts, d, f)) * f ** -0.5)
    cuts = [0, *np.sort(rng.integers(0, rows + 1, experts - 1)).tolist(), rows]
    return x, gu, dn, to(rng.standard_normal((rows, d))), cuts


@pytest.mark.parametrize("checkpoint", ["mx8", None])
@pytest.mark.parametrize("dtype,rows,experts,d,f", SIZES)
def test_gradients_at_kept_values(X, dtype, rows, experts, d, f, checkpoint):
    x, gu, dn, dy, cuts = inputs(dtype, rows, experts, d, f)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    leaves = [t.cuda().requires_grad_() for t in (x, gu, dn)]
    got = torch.autograd.grad(X.mlp(*leaves, off, checkpoint=checkpoint), leaves, dy.cuda())
    # the activation's input as the product gives it (its own tests say how near that is)
    h = f64(X.linear(x.cuda(), gu.cuda(), off))
    v = [f64(t) for t in (x, gu, dn, dy)]
    xk, hk = (kept(v[0], dtype, False), kept(h, dtype, True)) if checkpoint else (v[0], h)
    for g, want, name in zip(got, gradients(*v, h, cuts, dtype, xk, hk, hk), ("x", "w_gate_up", "w_down")):
        assert inside(f64(g), want), name
