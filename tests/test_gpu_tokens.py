"""Tokens sorted by expert and back on the GPU (sort_tokens, dispatch, combine
and the gradients) against plain numpy in float64, and a whole layer built of
the pieces."""

import numpy as np
import pytest
import torch

from oracle import mx as X

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


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def ref_order(ids, num_experts):
    flat = ids.reshape(-1).astype(np.int64)
    keep = np.flatnonzero((flat >= 0) & (flat < num_experts))
    src = keep[np.argsort(flat[keep], kind="stable")]
    row_src = np.full(flat.size, -1)
    row_src[:src.size] = src
    token_row = np.full(flat.size, -1)
    token_row[src] = np.arange(src.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=num_experts))])
    return offsets, row_src, token_row.reshape(ids.shape)


def some_ids(t, k, e, seed, kind="random"):
    rng = np.random.default_rng(seed)
    if kind == "random":      # distinct experts per token where there are enough
        return np.argsort(rng.random((t, e)), axis=1)[:, :k] if e >= k else rng.integers(0, e, (t, k))
    if kind == "same":        # one expert for everything, every pair a duplicate
        return np.full((t, k), e - 1)
    if kind == "dropped":     # a third of the choices name no expert, some tokens none at all
        ids = rng.integers(0, e, (t, k))
        ids[rng.random((t, k)) < 0.33] = -1
        ids[rng.random((t, k)) < 0.1] = e
        ids[rng.random(t) < 0.2] = -1
        return ids
    if kind == "none":
        return np.full((t, k), -1)
    if kind == "skew":        # expert 0 takes most, some experts nothing
        return np.minimum(rng.geometric(0.3, (t, k)) - 1, e - 1)
    raise ValueError(kind)


def assert_order(order, ids, num_experts):
    offsets, row_src, token_row = ref_order(ids, num_experts)
    assert np.array_equal(order.offsets.cpu().numpy(), offsets)
    assert np.array_equal(order.token_row.cpu().numpy(), token_row)
    assert np.array_equal(order.row_src.cpu().numpy(), row_src)


SIZES = [(1, 1, 1), (1, 16, 896), (3, 2, 5), (64, 1, 2), (65, 7, 1024), (256, 16, 896), (257, 16, 896), (700, 6, 3),
         (1000, 32, 64), (5000, 4, 1000), (8192, 16, 896), (70001, 2, 17)]


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("kind", ["random", "same", "dropped", "none", "skew"])
@pytest.mark.parametrize("t,k,e", SIZES)
def test_sort_matches_a_stable_sort(K, t, k, e, kind, dtype):
    ids = some_ids(t, k, e, t + 31 * k + e, kind)
    order = K.sort_tokens(torch.from_numpy(ids.astype(dtype)).cuda(), e)
    assert_order(order, ids, e)


def test_sort_the_largest_number_of_chunks(K):
    # more pairs than 512 chunks of the smallest size hold
    ids = some_ids(1 << 16, 32, 300, 5, "dropped")
    assert_order(K.sort_tokens(torch.from_numpy(ids).cuda(), 300), ids, 300)


def test_sort_ids_beyond_32_bits(K):
    ids = torch.tensor([[1 << 32, 3], [(1 << 33) + 2, -(1 << 32)], [2, 1]], device="cuda")
    assert_order(K.sort_tokens(ids, 4), np.array([[-1, 3], [-1, -1], [2, 1]]), 4)


def test_sort_of_a_view_and_of_nothing(K):
    ids = some_ids(50, 8, 20, 3)
    wide = torch.from_numpy(ids).cuda()
    assert_order(K.sort_tokens(wide[:, ::2], 20), ids[:, ::2], 20)
    assert_order(K.sort_tokens(wide[:0], 20), ids[:0], 20)


def case(t, k, e, d, dtype, kind, seed=0):
    """order, x, rows, w, dy and gradients of xs on the GPU, and their float64 copies"""
    g = torch.Generator().manual_seed(seed + t + d)
    ids = some_ids(t, k, e, seed + 1, kind)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    v = dict(x=rnd(t, d).to(DT[dtype]), rows=rnd(t * k, d).to(DT[dtype]), w=rnd(t, k), dy=rnd(t, d).to(DT[dtype]),
             dxs=rnd(t * k, d).to(DT[dtype]))
    return ids, {n: x.cuda() for n, x in v.items()}, {n: f64(x) for n, x in v.items()}


CASES = [(1, 16, 896, 7168, "bf16", "random"), (1, 1, 1, 1, "fp32", "random"), (5, 3, 4, 33, "bf16", "dropped"),
         (5, 3, 4, 33, "fp32", "dropped"), (9, 4, 2, 7, "fp16", "skew"), (40, 8, 64, 256, "fp16", "dropped"),
         (33, 32, 7, 1000, "fp32", "same"), (129, 6, 40, 2880, "bf16", "skew"), (300, 4, 1000, 136, "bf16", "none"),
         (257, 16, 896, 516, "fp32", "random"), (1200, 5, 60, 129, "bf16", "dropped"), (2050, 2, 9, 8, "fp16", "random")]


@pytest.mark.parametrize("t,k,e,d,dtype,kind", CASES)
def test_dispatch_and_its_gradient(K, t, k, e, d, dtype, kind):
    ids, v, r = case(t, k, e, d, dtype, kind)
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), e)
    x = v["x"].requires_grad_()
    xs = K.dispatch(x, order)
    offsets, row_src, token_row = ref_order(ids, e)
    ref = np.where(row_src[:, None] >= 0, r["x"][np.maximum(row_src, 0) // k], 0.0)
    assert np.array_equal(f64(xs), ref)
    dx, = torch.autograd.grad(xs, x, v["dxs"])
    terms = np.where(token_row[:, :, None] >= 0, r["dxs"][np.maximum(token_row, 0)], 0.0)
    assert dx.dtype == x.dtype
    assert_sum(dx, terms, dtype)


def assert_sum(got, terms, dtype):
    # terms [T, k, d]: k products (one rounding each, or fused) and k - 1
    # additions in fp32, at most 2k half steps of partial sums of magnitudes;
    # then one rounding to the type (fp16: 2^-25 for its smallest numbers)
    ref, mag, k = terms.sum(1), np.abs(terms).sum(1), terms.shape[1]
    bound = 2 * k * 2.0 ** -24 * mag
    bound += torch.finfo(DT[dtype]).eps / 2 * (np.abs(ref) + bound) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    bad = ~(np.abs(f64(got) - ref) <= bound)
    assert not bad.any(), np.argwhere(bad)[:5]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("t,k,e,d,dtype,kind", CASES)
def test_combine_and_its_gradients(K, t, k, e, d, dtype, kind, weighted):
    ids, v, r = case(t, k, e, d, dtype, kind, seed=50)
    offsets, row_src, token_row = ref_order(ids, e)
    # what no pair refers to is never read: rows behind the last and weights of dropped pairs hold NaN
    v["rows"][offsets[-1]:] = float("nan")
    v["w"][torch.from_numpy(token_row < 0).cuda()] = float("nan")
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), e)
    rows, w = v["rows"].requires_grad_(), v["w"].requires_grad_()
    y = K.combine(rows, w if weighted else None, order)
    there = token_row >= 0
    w64 = np.where(there, r["w"] if weighted else 1.0, 0.0)
    picked = np.where(there[:, :, None], r["rows"][np.maximum(token_row, 0)], 0.0)
    assert_sum(y, picked * w64[:, :, None], dtype)
    assert (f64(y)[~there.any(1)] == 0).all()
    grads = torch.autograd.grad(y, (rows, w) if weighted else (rows,), v["dy"])
    # drows: one product in fp32, rounded once more to the type (for fp32 it is the same rounding)
    dr = np.zeros((t * k, d))
    src = row_src[:offsets[-1]]
    dr[:offsets[-1]] = r["dy"][src // k] * w64.reshape(-1)[src][:, None]
    bound = (2.0 ** -24 + torch.finfo(DT[dtype]).eps) * np.abs(dr) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert (np.abs(f64(grads[0]) - dr) <= bound).all()
    assert (f64(grads[0])[offsets[-1]:] == 0).all()
    if weighted:
        # dw: d products and additions in fp32 in some fixed order
        dw = (picked * r["dy"][:, None, :]).sum(2)
        mag = (np.abs(picked) * np.abs(r["dy"][:, None, :])).sum(2)
        assert grads[1].dtype == torch.float32
        assert (np.abs(f64(grads[1]) - dw) <= 2 * d * 2.0 ** -24 * mag).all()
        assert (f64(grads[1])[~there] == 0).all()


def test_gradients_against_differences(K):
    # the sum over the outputs times fixed weights, moved along one random direction of each input, in fp32: the
    # operators are linear in each, so a central difference is exact up to the sums' rounding
    t, k, e, d = 30, 4, 6, 40
    ids, v, _ = case(t, k, e, d, "fp32", "dropped", seed=70)
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), e)
    x, w, gy = v["x"].requires_grad_(), v["w"].requires_grad_(), v["dy"]

    def loss(x, w):
        return (K.combine(K.dispatch(x, order) * 1.5, w, order).double() * gy.double()).sum()

    gx, gw = torch.autograd.grad(loss(x, w), (x, w))
    for i, (p, g) in enumerate(((x, gx), (w, gw))):
        u = torch.randn(p.shape, generator=torch.Generator().manual_seed(i)).cuda()
        args = lambda s: [q.detach() + s * u if q is p else q.detach() for q in (x, w)]  # noqa: E731
        diff = float((loss(*args(0.5)) - loss(*args(-0.5))))
        ref = float((g.double() * u.double()).sum())
        # k t d terms of order one, each off by a few 2^-24
        assert abs(diff - ref) <= 16 * 2.0 ** -24 * t * k * d * 6


def test_only_the_gradients_that_are_asked_for(K):
    t, k, e, d = 20, 3, 5, 64
    ids, v, _ = case(t, k, e, d, "bf16", "random", seed=80)
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), e)
    rows, w = v["rows"].requires_grad_(), v["w"].requires_grad_()
    both = torch.autograd.grad(K.combine(rows, w, order), (rows, w), v["dy"])
    assert torch.equal(torch.autograd.grad(K.combine(rows, w.detach(), order), rows, v["dy"])[0], both[0])
    assert torch.equal(torch.autograd.grad(K.combine(rows.detach(), w, order), w, v["dy"])[0], both[1])
    assert K.combine(rows.detach(), w.detach(), order).grad_fn is None


def test_an_order_changed_before_the_backward_pass_is_an_error(K):
    ids, v, _ = case(20, 3, 5, 64, "fp32", "random", seed=81)
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), 5)
    x, w = v["x"].requires_grad_(), v["w"].requires_grad_()
    xs, y = K.dispatch(x, order), K.combine(v["rows"], w, order)
    order.token_row.zero_()
    with pytest.raises(RuntimeError, match="inplace"):
        torch.autograd.grad(xs, x, v["dxs"])
    with pytest.raises(RuntimeError, match="inplace"):
        torch.autograd.grad(y, w, v["dy"])


def test_a_second_derivative_is_refused(K):
    ids, v, _ = case(20, 3, 5, 64, "fp32", "random", seed=82)
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), 5)
    x, w = v["x"].requires_grad_(), v["w"].requires_grad_()
    y = K.combine(K.dispatch(x, order), w, order)
    gx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gx.sum(), w)


def test_two_graphs_replayed_in_turn(K):
    # each capture has a workspace and buffers of its own (more pairs than one workgroup sorts)
    sets = []
    for i in range(2):
        ids, v, _ = case(1500, 8, 64, 40, "bf16", "dropped", seed=200 + i)
        ids = torch.from_numpy(ids).cuda()

        def step(ids=ids, v=v):
            order = K.sort_tokens(ids, 64)
            return order.row_src, K.combine(K.dispatch(v["x"], order), v["w"], order)

        ref = [o.clone() for o in step()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        sets.append((graph, out, ref, ids, v))  # (a graph reads its inputs: they live as long)
    for _ in range(3):
        for graph, *_ in sets:
            graph.replay()
        torch.cuda.synchronize()
        for _, out, ref, *_ in sets:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
        for _, out, *_ in sets:
            for o in out:
                o.zero_()


def test_broadcast_and_strided_inputs(K):
    t, k, e, d = 37, 4, 8, 48
    ids, v, r = case(t, k, e, d, "fp32", "dropped", seed=90)
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), e)
    rows, w = v["rows"].requires_grad_(), v["w"].requires_grad_()
    # y.sum(): an expanded gradient
    a = torch.autograd.grad(K.combine(rows, w, order).sum(), (rows, w))
    b = torch.autograd.grad(K.combine(rows, w, order), (rows, w), torch.ones(t, d, device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # a row shared by every token, rows inside a wider matrix, weights of a transposed one
    one = v["x"][:1].expand(t, d)
    assert torch.equal(K.dispatch(one, order), K.dispatch(one.contiguous(), order))
    lead = v["x"][:1].clone().requires_grad_()
    g, = torch.autograd.grad(K.dispatch(lead.expand(t, d), order), lead, v["dxs"])
    n = int(order.offsets[-1])
    # n additions in fp32, in two stages
    assert np.abs(f64(g)[0] - r["dxs"][:n].sum(0)).max() <= 2 * t * k * 2.0 ** -24 * np.abs(r["dxs"][:n]).sum(0).max()
    wide = torch.zeros(t * k, d + 7, device="cuda")
    wide[:, 3:3 + d] = rows.detach()
    wt = w.detach().t().contiguous().t()
    assert torch.equal(K.combine(wide[:, 3:3 + d], wt, order), K.combine(rows.detach(), w.detach(), order))
    xw = torch.zeros(t, d + 5, device="cuda")
    xw[:, 5:] = v["x"]
    assert torch.equal(K.dispatch(xw[:, 5:], order), K.dispatch(v["x"], order))


@pytest.mark.parametrize("dtype,cols", [(torch.uint8, 224), (torch.uint8, 7), (torch.int64, 3), (torch.int16, 10)])
def test_dispatch_moves_any_elements(K, dtype, cols):
    ids = some_ids(70, 4, 9, 1, "dropped")
    order = K.sort_tokens(torch.from_numpy(ids).cuda(), 9)
    x = torch.randint(0, 100, (70, cols)).to(dtype).cuda()
    row_src = ref_order(ids, 9)[1]
    ref = np.where(row_src[:, None] >= 0, x.cpu().numpy()[np.maximum(row_src, 0) // 4], 0)
    assert np.array_equal(K.dispatch(x, order).cpu().numpy(), ref)


def test_c_calls_leave_what_is_not_theirs(K):
    # without num_rows the rows that no pair has stay; entries of token_row outside the buffer are skipped
    from mxfp4_expert_grouped_amd import mxmoe as M
    t, k, d, cap = 3, 2, 40, 4
    token_row = torch.tensor([[0, 9], [-5, 2], [4, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    x = torch.randn(t, d, device="cuda")
    buf = torch.full((cap + 8, d), 1.5, device="cuda")
    M.moe_dispatch_rows(x.data_ptr(), 4 * d, 4 * d, token_row.data_ptr(), t, k, None, cap, buf.data_ptr(), 4 * d, st)
    ref = torch.full_like(buf, 1.5)
    ref[0], ref[2] = x[0], x[1]
    assert torch.equal(buf, ref)
    n = torch.tensor([3], dtype=torch.int32, device="cuda")
    M.moe_dispatch_rows(x.data_ptr(), 4 * d, 4 * d, token_row.data_ptr(), t, k, n.data_ptr(), cap, buf.data_ptr(), 4 * d, st)
    ref[3] = 0
    assert torch.equal(buf, ref)
    y = torch.empty(t, d, device="cuda")
    w = torch.randn(t, k, device="cuda")
    M.moe_combine_rows(buf.data_ptr(), M.MOE_SRC_FP32, cap, d, d, token_row.data_ptr(), w.data_ptr(), t, k, y.data_ptr(), d, st)
    assert torch.equal(y, torch.stack([w[0, 0] * buf[0], w[1, 1] * buf[2], torch.zeros(d, device="cuda")]))
    dr = torch.full((cap + 8, d), 2.5, device="cuda")
    dw = torch.empty(t, k, device="cuda")
    M.moe_combine_rows_backward(x.data_ptr(), buf.data_ptr(), M.MOE_SRC_FP32, cap, d, d, d, token_row.data_ptr(), w.data_ptr(),
                                t, k, None, dr.data_ptr(), d, dw.data_ptr(), st)
    ref = torch.full_like(dr, 2.5)
    ref[0], ref[2] = w[0, 0] * x[0], w[1, 1] * x[1]
    assert torch.equal(dr, ref)
    assert (dw[torch.tensor([[False, True], [True, False], [True, True]])] == 0).all() and (dw != 0).sum() == 2


@pytest.mark.parametrize("t,k,e,d", [(6, 4, 20, 256), (1500, 8, 64, 128)])
def test_forward_and_backward_in_a_replayed_graph(K, t, k, e, d):
    ids, v, _ = case(t, k, e, d, "bf16", "dropped", seed=99)
    ids = torch.from_numpy(ids).cuda()
    x0, w0 = v["x"], v["w"]

    def step():
        # leaves of its own in every call: no graph from outside the capture holds them
        x, w = x0.detach().requires_grad_(), w0.detach().requires_grad_()
        order = K.sort_tokens(ids, e)
        y = K.combine(K.dispatch(x, order) * 2, w, order)
        dx, dw = torch.autograd.grad(y, (x, w), v["dy"])
        # the same without autograd
        drows, dw2 = K.combine_backward(v["dy"], K.dispatch(x0, order) * 2, w0, order)
        return y.detach(), order.token_row, dx, dw, K.dispatch_backward(drows * 2, order), dw2

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x0.copy_(torch.randn_like(x0))
        w0.copy_(torch.rand_like(w0))
        ids.copy_(torch.from_numpy(some_ids(t, k, e, i, "dropped" if i % 2 else "skew")))
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        assert torch.equal(got[2], got[4]) and torch.equal(got[3], got[5])


def test_on_another_stream(K):
    ids, v, _ = case(400, 8, 50, 512, "bf16", "random", seed=7)
    ids = torch.from_numpy(ids).cuda()

    def step():
        order = K.sort_tokens(ids, 50)
        return K.combine(K.dispatch(v["x"], order), v["w"], order)

    ref = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in got)


def test_refusals(K):
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        K.sort_tokens(ids.float(), 4)
    with pytest.raises(ValueError):
        K.sort_tokens(ids[0], 4)
    with pytest.raises(ValueError):
        K.sort_tokens(ids.cpu(), 4)
    from mxfp4_expert_grouped_amd.mxmoe import MoeError
    for n in (0, 1025):
        with pytest.raises(MoeError):
            K.sort_tokens(ids, n)
    with pytest.raises(MoeError):
        K.sort_tokens(torch.zeros(4, 33, dtype=torch.int32, device="cuda"), 4)
    order = K.sort_tokens(ids, 4)
    with pytest.raises(ValueError):
        K.dispatch(torch.zeros(5, 8, device="cuda"), order)
    with pytest.raises(ValueError):
        K.dispatch(torch.zeros(4, 8), order)
    with pytest.raises(ValueError):
        K.dispatch(torch.zeros(4, 8, device="cuda", dtype=torch.float64, requires_grad=True), order)
    with pytest.raises(ValueError):
        K.combine(torch.zeros(8, 8, device="cuda", dtype=torch.float64), None, order)
    with pytest.raises(ValueError):
        K.combine(torch.zeros(7, 8, device="cuda"), None, order)
    with pytest.raises(ValueError):
        K.combine(torch.zeros(8, 8, device="cuda"), torch.zeros(4, 2, device="cuda", dtype=torch.bfloat16), order)
    with pytest.raises(ValueError):
        K.combine(torch.zeros(8, 8, device="cuda"), torch.zeros(4, 3, device="cuda"), order)


# ---------------------------------------------------------------------------
# a layer of the pieces
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("t,k,e,d,f", [(1, 4, 16, 256, 128), (50, 4, 16, 256, 128), (700, 2, 4, 512, 256), (9, 3, 5, 96, 64)])
def test_a_layer_of_the_pieces(K, t, k, e, d, f):
    # sort, quantise, dispatch codes and scales, gate_up, a GELU-gated activation of the caller's own, quantise,
    # down, combine; checked stage by stage in float64 on the GPU's own quantised operands
    from mxfp4_expert_grouped_amd import layer as L
    g = torch.Generator(device="cuda").manual_seed(t + d)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ids = torch.from_numpy(some_ids(t, k, e, t, "dropped" if t > 10 else "random")).cuda()
    x, w = rnd(t, d).bfloat16(), rnd(t, k).softmax(1)
    gu = [L.quantize_mx4(rnd(2 * f, d) * d ** -0.5) for _ in range(e)]
    dn = [L.quantize_mx4(rnd(d, f) * f ** -0.5) for _ in range(e)]
    st = lambda m, i: torch.stack([q[i] for q in m])  # noqa: E731
    order = K.sort_tokens(ids, e)
    xc, xsc = L.quantize_mx4(x)
    gate_up = L.linear_mx4(K.dispatch(xc, order), K.dispatch(xsc, order), st(gu, 0), st(gu, 1), offsets=order.offsets,
                           dtype=torch.float32)
    n = int(order.offsets[-1])
    h = torch.nn.functional.gelu(gate_up[:, :f]) * gate_up[:, f:]
    h[n:] = 0  # undefined rows: nothing of them may be a NaN block that a sum over all rows would meet
    hc, hs = L.quantize_mx4(h)
    o = L.linear_mx4(hc, hs, st(dn, 0), st(dn, 1), offsets=order.offsets, dtype=torch.float32)
    y = K.combine(o, w, order)

    dec = lambda q: X.mx_decode(q[0].cpu().numpy(), q[1].cpu().numpy(), "e2m1")  # noqa: E731
    offsets, row_src, token_row = ref_order(ids.cpu().numpy(), e)
    xq, hq = dec((xc, xsc)), dec((hc, hs))
    rgu, ro, mgu, mo = np.zeros((n, 2 * f)), np.zeros((n, d)), np.zeros((n, 2 * f)), np.zeros((n, d))
    for i in range(e):
        r = slice(offsets[i], offsets[i + 1])
        a = xq[row_src[r] // k]
        rgu[r], mgu[r] = a @ dec(gu[i]).T, np.abs(a) @ np.abs(dec(gu[i])).T
        ro[r], mo[r] = hq[r] @ dec(dn[i]).T, np.abs(hq[r]) @ np.abs(dec(dn[i])).T
    assert (np.abs(f64(gate_up)[:n] - rgu) <= (d + 1) * 2.0 ** -24 * mgu).all()
    bo = (f + 1) * 2.0 ** -24 * mo
    assert (np.abs(f64(o)[:n] - ro) <= bo).all()
    there, w64 = token_row >= 0, f64(w)
    wt = np.where(there, w64, 0.0)[:, :, None]
    if n:
        at = np.maximum(token_row, 0)
        ry = (wt * ro[at]).sum(1)
        assert (np.abs(f64(y) - ry) <= (wt * (bo + (2 * k + 1) * 2.0 ** -24 * mo)[at]).sum(1)).all()
