"""The standalone pieces of a sparse MoE layer with 4-bit weights, and how long they take.

Two groups of operators:

* MXFP4 (E2M1 elements, one E8M0 scale per 32 along the columns): quantisation
  of a matrix, the values its codes stand for, and the product of two such
  matrices, for one weight matrix or for one per expert with the rows sorted
  by expert;
* tokens sorted by expert and back: the order from the router's choices, a
  token's row copied to each of its experts, the experts' rows summed with the
  routing weights, and both gradients.

Widths are those of the repository's layer configurations (d_model 7168, d_ff
2048, gate and up together 4096, top-16 of 896 experts) where nothing else is
said.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token's activations, and back: latency
        dict(name="quantize_token", op="quantize", rows=1, cols=7168, dtype="bf16"),
        # a prompt's activations, a ragged number of tokens
        dict(name="quantize_activations", op="quantize", rows=8191, cols=7168, dtype="bf16"),
        # fp32 master weights of four experts' gate and up, at load time or for quantisation-aware training
        dict(name="quantize_weights", op="quantize", rows=16384, cols=7168, dtype="fp32"),
        # one token through a shared expert's gate and up projection, from its bf16 activations
        dict(name="linear_token", op="linear", rows=1, experts=0, used=0, n=4096, k=7168, skew=0.0, given="bf16", out="bf16"),
        # one token through its 16 experts' gate and up, of 64 experts on this GPU
        dict(name="experts_token", op="linear", rows=16, experts=64, used=16, n=4096, k=7168, skew=0.0, given="mx4", out="bf16"),
        # 256 decoded tokens over 64 experts: 64 rows each on average, uneven
        dict(name="experts_decode", op="linear", rows=4096, experts=64, used=64, n=4096, k=7168, skew=0.5, given="mx4", out="fp32"),
        # a prompt through a shared expert's gate and up, from its bf16 activations
        dict(name="linear_prompt", op="linear", rows=8192, experts=0, used=0, n=4096, k=7168, skew=0.0, given="bf16", out="bf16"),
        # a prompt of 8192 tokens through 64 experts' down projection, uneven, three experts without a row
        dict(name="experts_prompt", op="linear", rows=131072, experts=64, used=61, n=7168, k=2048, skew=0.25, given="mx4", out="bf16"),
        # 256 decoded tokens to their experts
        dict(name="dispatch_decode", op="dispatch", tokens=256, top_k=16, experts=896, d=7168, dtype="bf16", pad=0, backward=False),
        # a training step's batch to its experts and the gradient back, the last tokens padding
        dict(name="dispatch_train", op="dispatch", tokens=8192, top_k=16, experts=896, d=7168, dtype="bf16", pad=93, backward=True),
        # one token's experts summed: latency
        dict(name="combine_token", op="combine", tokens=1, top_k=16, experts=896, d=7168, dtype="bf16", pad=0, backward=False),
        # a training step's batch summed, with the gradients of the rows and of the routing weights, in fp32, a ragged batch
        dict(name="combine_train", op="combine", tokens=4095, top_k=16, experts=896, d=7168, dtype="fp32", pad=31, backward=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "dispatch", "combine"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=32 * _log(rng, 1, 224), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "linear":
        experts = rng.choice([0, 0, 1, _log(rng, 2, 96)])
        rows = _log(rng, 1, 16384)
        # widths of 32 to 7168, most in steps of 128, some of them odd for the tiles
        k = 128 * _log(rng, 1, 56) if rng.random() < 0.8 else 32 * _log(rng, 1, 64)
        n = 128 * _log(rng, 1, 56) if rng.random() < 0.7 else _log(rng, 1, 2048)
        used = experts if experts < 2 else min(rows, rng.randint(1, experts))
        return dict(op=op, rows=rows, experts=experts, used=used, n=n, k=k, skew=rng.choice([0.0, 0.5, 1.0]),
                    given=rng.choice(["bf16", "mx4"]), out=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    experts = _log(rng, 2, 896)
    tokens = _log(rng, 1, 4096)
    d = 8 * _log(rng, 4, 896) if rng.random() < 0.8 else _log(rng, 1, 2047)
    return dict(op=op, tokens=tokens, top_k=rng.randint(1, min(16, experts)), experts=experts, d=d,
                dtype=rng.choice(["bf16", "fp16", "fp32"]), pad=rng.choice([0, 0, tokens // 9, tokens // 2]),
                backward=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _counts(case, g):
    """Rows of each expert: every used one has at least one, the others are shared out by powers of a rank."""
    e, used, rows = case["experts"], case["used"], case["rows"]
    p = torch.arange(1, used + 1, device="cuda", dtype=torch.float64) ** -case["skew"]
    more = torch.floor(p / p.sum() * (rows - used)).long()
    more[0] += rows - used - more.sum()
    counts = torch.zeros(e, dtype=torch.int64, device="cuda")
    counts[torch.randperm(e, generator=g, device="cuda")[:used]] = more + 1
    return counts


def prepare(case, seed):
    g = _rng(seed)
    s = dict(case)
    if case["op"] == "quantize":
        # activations and weights are close to normal, with rows of different size
        gain = torch.exp(_normal((case["rows"], 1), g, 0.5))
        s["x"] = (_normal((case["rows"], case["cols"]), g) * gain).to(DTYPES[case["dtype"]])
        return s
    if case["op"] == "linear":
        e, n, k = max(1, case["experts"]), case["n"], case["k"]
        codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((e, n, k // 32), dtype=torch.uint8, device="cuda")
        for i in range(e):
            codes[i], scales[i] = _plain_quantize(_normal((n, k), g, k ** -0.5))
        x = _normal((case["rows"], k), g).to(torch.bfloat16)
        if case["given"] == "bf16":
            s["x"] = x
        else:
            s["codes"], s["scales"] = _plain_quantize(x)
        if case["experts"]:
            counts = _counts(case, g)
            offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
            offsets[1:] = counts.cumsum(0)
            s["offsets"] = offsets.to(torch.int32)
            # what a program that pads its groups knows of them beforehand
            s["active"] = counts.nonzero()[:, 0]
            s["most"] = int(counts.max())
            s["w_codes"], s["w_scales"] = codes, scales
        else:
            s["w_codes"], s["w_scales"] = codes[0], scales[0]
        return s
    t, k, e, d, dt = case["tokens"], case["top_k"], case["experts"], case["d"], DTYPES[case["dtype"]]
    # a router's choices: the top k of noisy logits with some experts hotter than others
    logits = _normal((t, e), g) + _normal((1, e), g, 0.5)
    top, ids = logits.topk(k, dim=1)
    s["ids"] = ids.sort(dim=1)[0]
    s["ids"][t - case["pad"]:] = -1  # padding tokens go to no expert
    if case["op"] == "dispatch":
        s["x"] = _normal((t, d), g).to(dt).requires_grad_(case["backward"])
        s["dxs"] = _normal((t * k, d), g).to(dt) if case["backward"] else None
    else:
        w = torch.sigmoid(top)
        s["w"] = (w / w.sum(1, keepdim=True)).requires_grad_(case["backward"])
        s["rows"] = _normal((t * k, d), g).to(dt).requires_grad_(case["backward"])
        s["dy"] = _normal((t, d), g).to(dt) if case["backward"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _power(e):
    """2^e as fp32, for whole e from -127 to 127."""
    return torch.where(e > -127, ((e + 127) << 23).view(torch.float32), torch.full((), 2.0 ** -127, device=e.device))


def _plain_quantize(x):
    """MXFP4 codes (element 2i in the low half of byte i) and scale bytes of a matrix's rows."""
    rows, cols = x.shape
    v = x.float().reshape(rows, cols // 32, 32)
    amax = v.abs().amax(2)
    e = torch.frexp(amax)[1].to(torch.int32) - 3
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    q = v * _power(-e)[:, :, None]
    m = q.abs()
    # E2M1 magnitudes 0 0.5 1 1.5 2 3 4 6: a value in the middle of two goes to the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75).to(torch.uint8) + (m > 1.25).to(torch.uint8) + (m >= 1.75).to(torch.uint8)
            + (m > 2.5).to(torch.uint8) + (m >= 3.5).to(torch.uint8) + (m > 5.0).to(torch.uint8))
    code = (code + 8 * torch.signbit(q).to(torch.uint8)).reshape(rows, cols // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _plain_values(codes, scales):
    """The fp32 values of MXFP4 codes [..., K/2] and scales [..., K/32]."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*scales.shape, 32)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    v = torch.where(c < 8, grid[(c & 7).int()], -grid[(c & 7).int()])
    return (v * _power(scales.int() - 127)[..., None]).reshape(*scales.shape[:-1], -1)


def _plain_linear(s, a):
    if not s["experts"]:
        return (a @ _plain_values(s["w_codes"], s["w_scales"]).T).to(DTYPES[s["out"]])
    # the experts that have rows, each one's rows padded to the longest
    w = _plain_values(s["w_codes"][s["active"]], s["w_scales"][s["active"]])
    starts = s["offsets"].long()[s["active"]]
    row = torch.arange(a.shape[0], device=a.device)
    group = torch.searchsorted(starts, row, right=True) - 1
    at = row - starts[group]
    padded = torch.zeros((w.shape[0], s["most"], a.shape[1]), device=a.device)
    padded[group, at] = a
    return torch.bmm(padded, w.transpose(1, 2))[group, at].to(DTYPES[s["out"]])


def _plain_order(ids, experts):
    """offsets [E+1], row_src [T*k] (-1 behind the last row), token_row [T, k] (-1 for a choice of no expert)."""
    flat = ids.reshape(-1)
    here = (flat >= 0) & (flat < experts)
    key, pair = torch.where(here, flat, torch.full_like(flat, experts)).sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=ids.device), right=False).to(torch.int32)
    row_src = torch.where(key < experts, pair, torch.full_like(pair, -1)).to(torch.int32)
    token_row = torch.empty_like(flat)
    token_row[pair] = torch.arange(flat.numel(), device=ids.device)
    token_row = torch.where(here, token_row, torch.full_like(flat, -1)).reshape(ids.shape).to(torch.int32)
    return offsets, row_src, token_row


def _plain_sum(rows, token_row, w):
    """sum over a token's rows, times their weights, in fp32."""
    r = rows.detach()[token_row.clamp(min=0)].float()
    r = torch.where((token_row >= 0)[:, :, None], r, torch.zeros((), device=rows.device))
    return r.sum(1) if w is None else (r * w.detach()[:, :, None]).sum(1)


def _plain_spread(x, row_src, top_k):
    """Row r is a copy of the row of its token, or zero where there is none."""
    r = x.detach()[(row_src // top_k).clamp(min=0).long()]
    return torch.where((row_src >= 0)[:, None], r, torch.zeros((), dtype=r.dtype, device=x.device))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quantize":
        return _plain_values(*_plain_quantize(s["x"])).to(s["x"].dtype)
    if s["op"] == "linear":
        codes, scales = _plain_quantize(s["x"]) if s["given"] == "bf16" else (s["codes"], s["scales"])
        return _plain_linear(s, _plain_values(codes, scales))
    offsets, row_src, token_row = _plain_order(s["ids"], s["experts"])
    if s["op"] == "dispatch":
        out = dict(offsets=offsets, row_src=row_src, token_row=token_row, xs=_plain_spread(s["x"], row_src, s["top_k"]))
        if s["backward"]:
            out["dx"] = _plain_sum(s["dxs"], token_row, None).to(s["x"].dtype)
        return out
    rows, w = s["rows"].detach(), s["w"].detach()
    out = dict(y=_plain_sum(rows, token_row, w).to(rows.dtype))
    if s["backward"]:
        dy = s["dy"].float()
        pair = row_src.clamp(min=0).long()
        drows = dy[pair // s["top_k"]] * w.reshape(-1)[pair][:, None]
        out["drows"] = torch.where((row_src >= 0)[:, None], drows, torch.zeros((), device=rows.device)).to(rows.dtype)
        dw = (rows[token_row.clamp(min=0)].float() * dy[:, None, :]).sum(2)
        out["dw"] = torch.where(token_row >= 0, dw, torch.zeros((), device=rows.device))
    return out


def _run_own(s):
    from mxfp4_expert_grouped_amd import layer, tokens

    if s["op"] == "quantize":
        codes, scales = layer.quantize_mx4(s["x"])
        return layer.dequantize_mx4(codes, scales, dtype=s["x"].dtype)
    if s["op"] == "linear":
        codes, scales = layer.quantize_mx4(s["x"]) if s["given"] == "bf16" else (s["codes"], s["scales"])
        return layer.linear_mx4(codes, scales, s["w_codes"], s["w_scales"],
                                offsets=s["offsets"] if s["experts"] else None, dtype=DTYPES[s["out"]])
    order = tokens.sort_tokens(s["ids"], s["experts"])
    if s["op"] == "dispatch":
        xs = tokens.dispatch(s["x"], order)
        out = dict(offsets=order.offsets, row_src=order.row_src, token_row=order.token_row, xs=xs)
        if s["backward"]:
            out["dx"], = torch.autograd.grad(xs, s["x"], s["dxs"])
        return out
    y = tokens.combine(s["rows"], s["w"], order)
    out = dict(y=y)
    if s["backward"]:
        out["drows"], out["dw"] = torch.autograd.grad(y, (s["rows"], s["w"]), s["dy"])
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "quantize":
        # read once, its values written once (the codes in between need not leave the chip)
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * SIZE[case["dtype"]], "flops": 0}
    if case["op"] == "linear":
        r, n, k = case["rows"], case["n"], case["k"]
        per = 0.5 + 1 / 32
        mats = case["used"] if case["experts"] else 1
        a = r * k * (2 if case["given"] == "bf16" else per)
        return {"bytes": int(mats * n * k * per + a + r * n * SIZE[case["out"]]), "flops": 2 * r * n * k}
    t, k, d, sz = case["tokens"], case["top_k"], case["d"], SIZE[case["dtype"]]
    pairs = (t - case["pad"]) * k
    order = t * k * (8 + 4 + 4)
    if case["op"] == "dispatch":
        n = (t + t * k) * d * sz
        return {"bytes": order + n * (2 if case["backward"] else 1), "flops": pairs * d if case["backward"] else 0}
    n = (pairs + t) * d * sz
    if case["backward"]:
        n += (t + t * k) * d * sz
    return {"bytes": order + n, "flops": pairs * d * (5 if case["backward"] else 2)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_codes(x):
    """Signed E2M1 values and block exponents in 64 bits, by the distance to every grid value."""
    rows, cols = x.shape
    v = x.double().reshape(-1, 32)
    amax = v.abs().max(1).values
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    # log2 may round up to a power that amax does not reach
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e) - 2
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    q = v / torch.exp2(e)[:, None]
    m = q.abs().clamp(max=6.0)
    # the step of the grid around m: 0.5 up to 2, 1 up to 4, then 2; torch.round sends halves to even
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    g = torch.round(m / step) * step
    return torch.where(torch.signbit(q), -g, g), e, (rows, cols)


def _exact_values(x):
    parts = []
    for block in x.split(max(1, (1 << 26) // x.shape[1])):
        g, e, shape = _exact_codes(block)
        parts.append((g * torch.exp2(e)[:, None]).reshape(shape))
    return torch.cat(parts)


def _exact_decode(codes, scales):
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    v[:, 0::2] = value[(codes % 16).long()]
    v[:, 1::2] = value[torch.div(codes, 16, rounding_mode="floor").long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_values(s["x"])
    if case["op"] == "linear":
        if case["given"] == "bf16":
            a = _exact_values(s["x"])
        else:
            a = _exact_decode(s["codes"], s["scales"])
        if not case["experts"]:
            return a @ _exact_decode(s["w_codes"], s["w_scales"]).T
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        o = s["offsets"].tolist()
        for e in range(case["experts"]):
            if o[e] < o[e + 1]:
                y[o[e]:o[e + 1]] = a[o[e]:o[e + 1]] @ _exact_decode(s["w_codes"][e], s["w_scales"][e]).T
        return y
    t, k, e, d = case["tokens"], case["top_k"], case["experts"], case["d"]
    flat = s["ids"].reshape(-1).cpu()
    pairs = sorted((int(v), p) for p, v in enumerate(flat.tolist()) if 0 <= v < e)
    row_src = torch.full((t * k,), -1, dtype=torch.int64)
    token_row = torch.full((t * k,), -1, dtype=torch.int64)
    at = torch.tensor([p for _, p in pairs], dtype=torch.int64)
    row_src[: len(pairs)] = at
    token_row[at] = torch.arange(len(pairs))
    counts = torch.bincount(flat[(flat >= 0) & (flat < e)], minlength=e)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    at, n = at.cuda(), len(pairs)
    token = torch.div(at, k, rounding_mode="floor")
    if case["op"] == "dispatch":
        xs = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
        xs[:n] = s["x"].detach()[token].double()
        out = dict(offsets=offsets.int(), row_src=row_src.int(), token_row=token_row.reshape(t, k).int(), xs=xs)
        if case["backward"]:
            out["dx"] = torch.zeros(t, d, dtype=torch.float64, device="cuda").index_add_(0, token, s["dxs"][:n].double())
        return out
    rows, w = s["rows"].detach()[:n].double(), s["w"].detach().reshape(-1)[at].double()
    out = dict(y=torch.zeros(t, d, dtype=torch.float64, device="cuda").index_add_(0, token, rows * w[:, None]))
    if case["backward"]:
        dy = s["dy"][token].double()
        out["drows"] = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
        out["drows"][:n] = dy * w[:, None]
        dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dw[at] = (rows * dy).sum(1)
        out["dw"] = dw.reshape(t, k)
    return out
