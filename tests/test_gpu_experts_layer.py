"""The experts' operators as a layer on the GPU: the network, its gradients
through autograd, captured graphs, other streams, equal bytes of equal calls,
and tensors past 32 bits."""

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
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def X():
    from mxfp4_expert_grouped_amd import experts
    return experts


@pytest.fixture(scope="module")
def K():
    from mxfp4_expert_grouped_amd import tokens
    return tokens


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b)) and len(a) == len(b)


def inputs(t, top_k, e, d, f, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ids = torch.rand((t, e), generator=g, device="cuda").topk(top_k, dim=1)[1]
    ids[t - t // 9:] = -1  # padding
    return dict(ids=ids, x=rnd(t, d).to(dtype), gu=(rnd(e, 2 * f, d) * d ** -0.5).to(dtype), dn=(rnd(e, d, f) * f ** -0.5).to(dtype),
                weights=torch.rand((t, top_k), generator=g, device="cuda"), dy=rnd(t, d).to(dtype))


def plain(X, K, v, checkpoint):
    """the layer and its gradients by the functions without autograd"""
    order = K.sort_tokens(v["ids"], v["gu"].shape[0])
    at = order.offsets
    xs = K.dispatch(v["x"], order)
    h = X.linear(xs, v["gu"], at)
    a, kept_h = X.swiglu_keep(h) if checkpoint else (X.swiglu(h), h)
    o = X.linear(a, v["dn"], at)
    y = K.combine(o, v["weights"], order)
    do, dweights = K.combine_backward(v["dy"], o, v["weights"], order)
    da, _ = X.linear_backward(do, None, v["dn"], at, need_w=False)
    dh, a = X.swiglu_backward(da, kept_h, need_a=True)
    _, ddn = X.linear_backward(do, a, None, at, need_x=False)
    dxs, dgu = X.linear_backward(dh, X.quantize_mx8(xs) if checkpoint else xs, v["gu"], at)
    return y, K.dispatch_backward(dxs, order), dgu, ddn, dweights


def by_autograd(X, K, v, checkpoint, leaves=("x", "gu", "dn", "weights")):
    p = {n: v[n].detach().clone().requires_grad_(n in leaves) for n in ("x", "gu", "dn", "weights")}
    order = K.sort_tokens(v["ids"], v["gu"].shape[0])
    o = X.mlp(K.dispatch(p["x"], order), p["gu"], p["dn"], order.offsets, checkpoint=checkpoint)
    y = K.combine(o, p["weights"], order)
    got = torch.autograd.grad(y, [p[n] for n in leaves], v["dy"]) if leaves else ()
    by = dict(zip(leaves, got))
    return y.detach(), by.get("x"), by.get("gu"), by.get("dn"), by.get("weights")


@pytest.mark.parametrize("checkpoint", [None, "mx8"])
@pytest.mark.parametrize("t,top_k,e,d,f,dtype", [(64, 4, 10, 256, 128, torch.bfloat16), (300, 2, 5, 100, 33, torch.float16),
                                                 (9, 1, 3, 7, 5, torch.bfloat16), (2000, 6, 40, 512, 96, torch.bfloat16)])
def test_the_layer_through_autograd_is_the_functions(X, K, t, top_k, e, d, f, dtype, checkpoint):
    v = inputs(t, top_k, e, d, f, dtype, t)
    want = plain(X, K, v, checkpoint)
    assert same(by_autograd(X, K, v, checkpoint), want)
    # gradients of some only: the others are not computed, these stay
    for leaves in (("x",), ("gu",), ("dn",), ("gu", "dn"), ("x", "dn"), ("weights",), ()):
        got = by_autograd(X, K, v, checkpoint, leaves)
        for g, w, n in zip(got, want, ("y", "x", "gu", "dn", "weights")):
            assert torch.equal(g, w) if n == "y" or n in leaves else g is None


def test_the_layer_against_float64(X, K):
    v = inputs(48, 3, 6, 64, 32, seed=5)
    p = {n: v[n].double().requires_grad_() for n in ("x", "gu", "dn", "weights")}
    y = torch.zeros(48, 64, dtype=torch.float64, device="cuda")
    for t in range(48):
        for j in range(3):
            e = int(v["ids"][t, j])
            if e < 0:
                continue
            h = p["gu"][e] @ p["x"][t]
            y = y.index_add(0, torch.tensor([t], device="cuda"), (p["weights"][t, j] * (p["dn"][e] @ (torch.nn.functional.silu(h[:32]) * h[32:])))[None])
    ref = (y.detach(), *torch.autograd.grad(y, [p[n] for n in ("x", "gu", "dn", "weights")], v["dy"].double()))
    # bf16 rounds h, a, o, y and their gradients: at most seven roundings of 2^-8 relative to the size of what is
    # rounded lie between an input and a result; whatever the path, 16 times 2^-8 of the result's norm bounds their sum
    for got, want in zip(by_autograd(X, K, v, None), ref):
        assert float((got.double() - want).norm() / want.norm()) <= 16 * 2.0 ** -8
    # kept in 8 bits: a kept value is off by at most 2^-4, and by 2^-4 / sqrt(3) in the mean square; it enters a
    # gradient of gate and up through two factors, and x's once more
    for got, want in zip(by_autograd(X, K, v, "mx8"), ref):
        assert float((got.double() - want).norm() / want.norm()) <= 16 * 2.0 ** -8 + 3 * 2.0 ** -4


def test_products_are_adjoint(X):
    # <dy, x W^T> = <x, dy W> = <W, dy^T x>: the gradients of the forward pass that there is
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, dy = rnd(333, 200), rnd(7, 120, 200), rnd(333, 120)
    off = torch.tensor([0, 50, 50, 130, 131, 200, 300, 333], dtype=torch.int32, device="cuda")
    y, (dx, dw) = X.linear(x, w, off), X.linear_backward(dy, x, w, off)
    three = [(a.double() * b.double()) for a, b in ((dy, y), (x, dx), (w, dw))]
    # each result is off by half a step, 2^-8 of itself (the fp32 sums before it by much less)
    slack = sum(float(t.abs().sum()) for t in three) * 1.01 * 2.0 ** -8
    sums = [float(t.sum()) for t in three]
    assert max(sums) - min(sums) <= slack


def test_captured_calls_and_replays(X):
    v = inputs(200, 2, 6, 136, 40, seed=3)
    off = torch.tensor([0, 20, 20, 100, 101, 300, 350], dtype=torch.int32, device="cuda")
    x, do = v["x"].repeat(2, 1)[:350].clone(), v["dy"].repeat(2, 1)[:350].clone()
    odd_x, odd_w = x[:, :131].contiguous(), v["gu"][:, :, :131].contiguous()

    def run():
        h = X.linear(x, v["gu"], off)
        a, kept = X.swiglu_keep(h)
        y = X.linear(a, v["dn"], off)
        da, _ = X.linear_backward(do, None, v["dn"], off, need_w=False)
        dh, again = X.swiglu_backward(da, kept, need_a=True)
        return (y, *X.linear_backward(dh, X.quantize_mx8(x), v["gu"], off), X.linear_backward(do, again, None, off, need_x=False, w_dtype=torch.float32)[1],
                X.linear(odd_x, odd_w, off), *X.linear_backward(h, odd_x, odd_w, off))

    run()
    graphs = []
    for _ in range(2):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for i in range(4):
        # other rows, other groups, the graphs in turn, eager work in between
        x.copy_(torch.randn_like(x))
        do.copy_(torch.randn_like(do))
        odd_x.copy_(x[:, :131])
        off.copy_(torch.tensor([0, 20 + i, 20 + i, 100, 101, 300, 350 - 30 * i], dtype=torch.int32))
        want = run()
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert same(out, want)


def test_a_captured_training_step(X):
    v = inputs(64, 2, 4, 64, 32, seed=9)
    off = torch.tensor([0, 10, 30, 30, 64], dtype=torch.int32, device="cuda")
    x, dy = v["x"].clone(), v["dy"].clone()

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, v["gu"], v["dn"])]
        y = X.mlp(*leaves, off, checkpoint="mx8")
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(torch.randn_like(x))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want)


def test_another_stream(X):
    v = inputs(500, 2, 4, 512, 128, seed=4)
    off = torch.tensor([0, 100, 300, 450, 500], dtype=torch.int32, device="cuda")
    want = X.mlp(v["x"], v["gu"], v["dn"], off)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = v["x"] * 1  # made on that stream: a call elsewhere would not wait for it
        for _ in range(50):
            x = x * 1
        got = X.mlp(x, v["gu"], v["dn"], off)
    s.synchronize()
    assert torch.equal(got, want)
    # two at once, each with its own workspace
    many = [torch.cuda.Stream() for _ in range(3)]
    odd = v["gu"][:, :, :509].contiguous()
    xo = v["x"][:, :509].contiguous()
    want = (X.linear(xo, odd, off), *X.linear_backward(v["x"][:, :256].contiguous(), xo, odd, off))
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for st in many:
            with torch.cuda.stream(st):
                outs.append((X.linear(xo, odd, off), *X.linear_backward(v["x"][:, :256].contiguous(), xo, odd, off)))
    torch.cuda.synchronize()
    assert all(same(o, want) for o in outs)


def test_equal_calls_give_equal_bytes(X):
    v = inputs(3000, 2, 6, 640, 200, seed=6)
    off = torch.tensor([0, 900, 901, 1500, 1500, 2600, 3000], dtype=torch.int32, device="cuda")
    first = (X.linear(v["x"], v["gu"], off), *X.linear_backward(X.linear(v["x"], v["gu"], off), v["x"], v["gu"], off))
    long = v["x"][:, :96].contiguous(), v["x"][:, 96:196].contiguous()  # few results of long sums
    split = X.linear_backward(*long, None, None, need_x=False)[1]
    for _ in range(10):
        assert same((X.linear(v["x"], v["gu"], off), *X.linear_backward(X.linear(v["x"], v["gu"], off), v["x"], v["gu"], off)), first)
        assert torch.equal(X.linear_backward(*long, None, None, need_x=False)[1], split)


def test_what_autograd_saved_may_not_change(X):
    v = inputs(16, 1, 2, 32, 8)
    off = torch.tensor([0, 7, 16], dtype=torch.int32, device="cuda")
    w = v["gu"].requires_grad_()
    for changed in ("x", "offsets"):
        x, at = v["x"].clone(), off.clone()
        y = X.linear(x, w, at)
        (x if changed == "x" else at).zero_()
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()
    # in 8 bits x is no longer needed
    x = v["x"].clone()
    y = X.linear(x, w, off, checkpoint="mx8")
    want = X.linear_backward(torch.ones_like(y), X.quantize_mx8(x), None, off, need_x=False)[1]
    x.zero_()
    assert torch.equal(torch.autograd.grad(y.sum(), w)[0], want)


def test_gradients_once_only(X):
    x = torch.randn(8, 16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    w = torch.randn(8, 16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    for y in (X.linear(x, w), X.swiglu(x), X.mlp(x, w, torch.randn(16, 4, device="cuda", dtype=torch.bfloat16))):
        g, = torch.autograd.grad(y.sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()


def checked_rows(got, x, w, rows):
    # bf16 has 8 significant bits: half a step is 2^-8 of the value (finfo.eps / 2)
    want = x[rows].double() @ w.double().T
    mag = x[rows].double().abs() @ w.double().abs().T
    err = (got[rows].double() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + x.shape[1] * 2.0 ** -23 * 1.01 * mag).all())


def test_rows_and_results_past_32_bits(X):
    # x of 5 GB, y of 4.7 GB
    rows, n, k = 600011, 3904, 4160
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 15):
        part.normal_()
    w = torch.randn(2, n, k, device="cuda").bfloat16()
    off = torch.tensor([5, 299999, rows], dtype=torch.int32, device="cuda")
    y = X.linear(x, w, off)
    assert not y[:5].any()
    for e, at in ((0, [5, 6, 1000, 299998]), (1, [299999, 300000, 520000, rows - 1])):
        checked_rows(y, x, w[e], torch.tensor(at, device="cuda"))
    # and backwards: dx from y's size, dw over all rows
    dx, dw = X.linear_backward(y, x, w, off)
    assert not dx[:5].any()
    for e, at in ((0, [5, 1000, 299998]), (1, [299999, 520000, rows - 1])):
        checked_rows(dx, y, w[e].T, torch.tensor(at, device="cuda"))
    cols = torch.tensor([0, 1, 2000, n - 1], device="cuda")
    for e, (a, b) in enumerate(((5, 299999), (299999, rows))):
        want, mag = 0, 0
        for i in range(a, b, 1 << 15):
            yy, xx = y[i:min(b, i + (1 << 15))][:, cols].double(), x[i:min(b, i + (1 << 15))].double()
            want, mag = want + yy.T @ xx, mag + yy.abs().T @ xx.abs()
        assert bool(((dw[e][cols].double() - want).abs() <= 2.0 ** -8 * want.abs() + (b - a) * 2.0 ** -23 * 1.01 * mag).all())


def test_weights_past_32_bits(X):
    mats, n, k = 40, 8200, 8192  # 5.4 GB
    w = torch.empty(mats, n, k, dtype=torch.bfloat16, device="cuda")
    for part in w:
        part.normal_()
    for rows in (70, 3000):  # straight from memory and in tiles
        x = torch.randn(rows, k, device="cuda").bfloat16()
        off = torch.tensor([0] * (mats - 2) + [rows // 3, rows // 2, rows], dtype=torch.int32, device="cuda")
        y = X.linear(x, w, off)
        at = torch.tensor([rows // 3, rows // 2 - 1], device="cuda")
        checked_rows(y, x, w[mats - 2], at)
        checked_rows(y, x, w[mats - 1], torch.tensor([rows // 2, rows - 1], device="cuda"))
        dy = torch.randn(rows, n, device="cuda").bfloat16()
        dx, dw = X.linear_backward(dy, x, w, off)
        checked_rows(dx, dy, w[mats - 1].T, torch.tensor([rows // 2, rows - 1], device="cuda"))
        a = rows // 2
        checked_rows(dw[mats - 1], dy[a:].T.contiguous(), x[a:].T.contiguous(), torch.tensor([0, 4000, n - 1], device="cuda"))
        assert not dw[:mats - 3].any()
        del dw


def test_activations_past_32_bits(X):
    rows, f = 600007, 2048  # h of 4.9 GB, codes of 2.4 GB
    h = torch.empty(rows, 2 * f, dtype=torch.bfloat16, device="cuda")
    for part in h.split(1 << 15):
        part.normal_()
    da = h[:, :f] * 0.5
    a, kept = X.swiglu_keep(h)
    dh, again = X.swiglu_backward(da, kept, need_a=True)
    at = torch.tensor([0, 1, 262143, 262144, 524287, 524288, rows - 1], device="cuda")
    few_a, few_kept = X.swiglu_keep(h[at])
    assert torch.equal(a[at], few_a) and torch.equal(kept[0][at], few_kept[0]) and torch.equal(kept[1][at], few_kept[1])
    assert same([t[at] for t in (dh, again)], X.swiglu_backward(da[at], few_kept, need_a=True))


def test_more_pieces_than_a_launch_takes(X):
    rows = (1 << 29) + 5  # four pieces for a row of one column: past 2^31 of them
    v = torch.arange(rows, device="cuda", dtype=torch.int32).remainder_(509).to(torch.bfloat16)[:, None]
    codes, scales = X.quantize_mx8(v)
    few = X.quantize_mx8(v[:509].contiguous())
    back = X.dequantize_mx8(codes, scales)
    want = X.dequantize_mx8(*few)
    for start in (0, 509 * (1 << 19), rows // 509 * 509 - 509):
        assert torch.equal(codes[start:start + 509], few[0]) and torch.equal(scales[start:start + 509], few[1])
        assert torch.equal(back[start:start + 509], want)
    assert torch.equal(back[rows // 509 * 509:], want[:rows % 509])
