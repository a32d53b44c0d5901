"""Training and serving experts in 16 bits, and how long their operators take.

Two groups of operators:

* the product of rows sorted by expert with 16-bit expert matrices, for one
  matrix or for one per expert, ragged, with the gradients of both operands;
  on request the rows that the weights' gradient needs are kept in MXFP8 (E4M3
  elements, one E8M0 scale per 32 along the columns) instead of their own type;
* the gated activation between the two projections, silu(gate) * up, with its
  gradient; its input can be kept in MXFP8 for the backward pass too.

Widths are those of the repository's layer configurations (d_model 7168, d_ff
2048, gate and up together 4096) where nothing else is said.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32  # columns that share a scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    lin = dict(op="linear", n=4096, k=7168, dtype="bf16", kept="", backward=False)
    return [
        # one decoded token through a shared expert's gate and up projection: latency
        dict(lin, name="linear_token", rows=1, experts=0, used=0, skew=0.0),
        # one decoded token through its 16 experts' gate and up, of 64 experts on this GPU
        dict(lin, name="experts_token", rows=16, experts=64, used=16, skew=0.0),
        # 256 decoded tokens over 64 experts: 64 rows each on average, uneven
        dict(lin, name="experts_decode", rows=4096, experts=64, used=64, skew=0.5, dtype="fp16"),
        # a prompt through a shared expert's gate and up
        dict(lin, name="linear_prompt", rows=8192, experts=0, used=0, skew=0.0),
        # a prompt of 4096 tokens through 64 experts' down projection, uneven, three experts without a row
        dict(lin, name="experts_prompt", rows=65536, experts=64, used=61, skew=0.25, n=7168, k=2048),
        # a training step's gate and up: the product and both gradients
        dict(lin, name="experts_train", rows=32768, experts=64, used=64, skew=0.25, backward=True),
        # the same over fewer experts, the tokens' rows kept in 8 bits until the backward pass
        dict(lin, name="experts_train_kept8", rows=32768, experts=32, used=32, skew=0.25, kept="mx8", backward=True),
        # small experts of odd widths, in training, two of them without a row
        dict(lin, name="experts_train_odd", rows=5003, experts=13, used=11, skew=0.5, n=1031, k=509, dtype="fp16", backward=True),
        # one decoded token's 16 rows through the activation: latency
        dict(name="swiglu_token", op="swiglu", rows=16, d_ff=2048, dtype="bf16", kept="", backward=False),
        # a training step's rows, their gate and up kept in 8 bits until the backward pass
        dict(name="swiglu_train_kept8", op="swiglu", rows=131072, d_ff=2048, dtype="bf16", kept="mx8", backward=True),
        # the same with gate and up kept as they are
        dict(name="swiglu_train", op="swiglu", rows=32768, d_ff=2048, dtype="fp16", kept="", backward=True),
        # fp32 activations of an odd width, whose last block of a row is short
        dict(name="swiglu_train_odd", op="swiglu", rows=8191, d_ff=1365, dtype="fp32", kept="mx8", backward=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.3:
        return dict(op="swiglu", rows=_log(rng, 1, 65536), d_ff=32 * _log(rng, 1, 64) if rng.random() < 0.6 else _log(rng, 1, 2047),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), kept=rng.choice(["", "mx8", "mx8"]), backward=rng.random() < 0.7)
    # widths up to 7168, most in steps of 128, some of them odd for the tiles and for 16-byte pieces
    k = 128 * _log(rng, 1, 56) if rng.random() < 0.7 else _log(rng, 1, 2048)
    n = 128 * _log(rng, 1, 56) if rng.random() < 0.7 else _log(rng, 1, 2048)
    experts = rng.choice([0, 1, _log(rng, 2, 96), _log(rng, 2, 96)])
    experts = min(experts, 64 * 4096 * 7168 // (n * k))
    rows = min(_log(rng, 1, 32768), 32768 * 4096 * 7168 // (n * k))
    used = experts if experts < 2 else min(rows, rng.randint(1, experts))
    backward = rng.random() < 0.6
    return dict(op="linear", rows=rows, experts=experts, used=used, skew=rng.choice([0.0, 0.25, 0.5]), n=n, k=k,
                dtype=rng.choice(["bf16", "bf16", "fp16"]), kept=rng.choice(["", "mx8"]) if backward else "", backward=backward)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


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
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s, dt, rows = dict(case), DTYPES[case["dtype"]], case["rows"]
    # activations are close to normal, with rows of different size
    gain = torch.exp(_normal((rows, 1), g, 0.5))
    if case["op"] == "swiglu":
        s["h"] = (_normal((rows, 2 * case["d_ff"]), g, 1.5) * gain).to(dt).requires_grad_(case["backward"])
        s["da"] = _normal((rows, case["d_ff"]), g).to(dt) if case["backward"] else None
        return s
    e, n, k = case["experts"], case["n"], case["k"]
    w = torch.empty((max(1, e), n, k), dtype=dt, device="cuda")
    for i in range(max(1, e)):
        w[i] = _normal((n, k), g, k ** -0.5).to(dt)
    s["w"] = (w if e else w[0]).requires_grad_(case["backward"])
    s["x"] = (_normal((rows, k), g) * gain).to(dt).requires_grad_(case["backward"])
    s["dy"] = _normal((rows, n), g, n ** -0.5).to(dt) if case["backward"] else None
    if e:
        counts = _counts(case, g)
        offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = counts.cumsum(0)
        s["offsets"] = offsets.to(torch.int32)
        # what a program that pads its groups knows of them beforehand
        s["active"] = counts.nonzero()[:, 0]
        s["most"] = int(counts.max())
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _power(e):
    """2^e as fp32, for whole e from -127 to 127."""
    return torch.where(e > -127, ((e + 127) << 23).view(torch.float32), torch.full((), 2.0 ** -127, device=e.device))


def _plain_kept(v):
    """The values that MXFP8 codes of the rows of v (fp32) stand for: the largest magnitude m of 32 columns
    (fewer at the end of a row) gives 2^e, e = floor(log2 m) - 8, and v / 2^e is rounded to E4M3, at most 448."""
    rows, cols = v.shape
    blocks = -(-cols // BLOCK)
    p = torch.nn.functional.pad(v, (0, blocks * BLOCK - cols)).reshape(rows, blocks, BLOCK)
    amax = p.abs().amax(2)
    e = torch.frexp(amax)[1].to(torch.int32) - 9
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    q = p * _power(-e)[:, :, None]
    # E4M3 has three bits behind the first from 2^-6 on, and steps of 2^-9 below
    step = _power((torch.frexp(q)[1].to(torch.int32) - 4).clamp(min=-9))
    q = torch.where(q == 0, q, (torch.round(q / step) * step).clamp(-448.0, 448.0))
    return (q * _power(e)[:, :, None]).reshape(rows, blocks * BLOCK)[:, :cols]


def _plain_linear(s):
    dt, w, x = DTYPES[s["dtype"]], s["w"].detach().float(), s["x"].detach().float()
    if s["backward"]:
        dy = s["dy"].float()
        # what is kept is read back in its type
        xk = _plain_kept(x).to(dt).float() if s["kept"] else x
    if not s["experts"]:
        out = dict(y=(x @ w.T).to(dt))
        if s["backward"]:
            out["dx"], out["dw"] = (dy @ w).to(dt), (dy.T @ xk).to(dt)
        return out
    # the experts that have rows, each one's rows padded to the longest
    wa = w[s["active"]]
    starts = s["offsets"].long()[s["active"]]
    row = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(starts, row, right=True) - 1
    at = row - starts[group]

    def padded(a):
        p = torch.zeros((wa.shape[0], s["most"], a.shape[1]), device=a.device)
        p[group, at] = a
        return p

    out = dict(y=torch.bmm(padded(x), wa.transpose(1, 2))[group, at].to(dt))
    if s["backward"]:
        pdy = padded(dy)
        out["dx"] = torch.bmm(pdy, wa)[group, at].to(dt)
        out["dw"] = torch.zeros(w.shape, dtype=dt, device=w.device)
        out["dw"][s["active"]] = torch.bmm(pdy.transpose(1, 2), padded(xk)).to(dt)
    return out


def _plain_swiglu(s):
    h = s["h"].detach().float()
    dt, f = DTYPES[s["dtype"]], s["d_ff"]
    g, u = h[:, :f], h[:, f:]
    out = dict(a=(g / (1 + torch.exp(-g)) * u).to(dt))
    if s["backward"]:
        if s["kept"]:
            g, u = _plain_kept(g), _plain_kept(u)
        da, p = s["da"].float(), 1 / (1 + torch.exp(-g))
        dg = da * u * p * (1 + g * (1 - p))
        out["dh"] = torch.cat((dg, da * g * p), dim=1).to(dt)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return _plain_linear(s) if s["op"] == "linear" else _plain_swiglu(s)


def _run_own(s):
    from mxfp4_expert_grouped_amd import experts

    kept = s["kept"] or None
    if s["op"] == "swiglu":
        a = experts.swiglu(s["h"], checkpoint=kept)
        out = dict(a=a)
        if s["backward"]:
            out["dh"], = torch.autograd.grad(a, s["h"], s["da"])
        return out
    y = experts.linear(s["x"], s["w"], s["offsets"] if s["experts"] else None, checkpoint=kept)
    out = dict(y=y)
    if s["backward"]:
        out["dx"], out["dw"] = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    r, sz = case["rows"], SIZE[case["dtype"]]
    if case["op"] == "swiglu":
        f = case["d_ff"]
        # gate, up and the result; then the result's gradient and those of gate and up (what is kept in between is not counted)
        n = 3 * r * f + (3 * r * f if case["backward"] else 0)
        return {"bytes": n * sz, "flops": r * f * (16 if case["backward"] else 5)}
    n, k = case["n"], case["k"]
    mats = case["used"] if case["experts"] else 1
    total = mats * n * k + r * k + r * n
    if case["backward"]:
        total += r * n + r * k + max(1, case["experts"]) * n * k
    return {"bytes": total * sz, "flops": 2 * r * n * k * (3 if case["backward"] else 1)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_kept(x):
    """The MXFP8 values of x's rows in 64 bits, row pieces of 32 columns one by one, by the grid's own spacing."""
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        v = x[:, c:c + BLOCK]
        amax = v.abs().max(1).values
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
        # log2 may round up to a power that amax does not reach
        e = torch.where(torch.exp2(e) > amax, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e) - 8
        unit = torch.exp2(torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127)))[:, None]
        m = (v / unit).abs().clamp(max=448.0)
        spacing = torch.full_like(m, 2.0 ** -9)
        for i in range(-5, 9):
            spacing = torch.where(m >= 2.0 ** i, torch.full_like(m, 2.0 ** (i - 3)), spacing)
        out[:, c:c + BLOCK] = torch.copysign(torch.round(m / spacing) * spacing, v) * unit
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "swiglu":
        h, f = s["h"].detach().double(), case["d_ff"]
        out = dict(a=h[:, :f] * torch.sigmoid(h[:, :f]) * h[:, f:])
        if case["backward"]:
            if case["kept"]:
                h = torch.cat((_exact_kept(h[:, :f]), _exact_kept(h[:, f:])), dim=1)
            g, u, da = h[:, :f], h[:, f:], s["da"].double()
            p, q = torch.sigmoid(g), torch.sigmoid(-g)
            out["dh"] = torch.cat((da * u * (p + g * p * q), da * (g * p)), dim=1)
        return out
    n, k, rows = case["n"], case["k"], case["rows"]
    x, w = s["x"].detach(), s["w"].detach()
    w = w if case["experts"] else w[None]
    o = s["offsets"].tolist() if case["experts"] else [0, rows]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = dict(y=new(rows, n))
    if case["backward"]:
        out["dx"], out["dw"] = new(rows, k), new(*w.shape)
    for e in range(len(o) - 1):
        a, b = o[e], o[e + 1]
        if a == b:
            continue
        we, xe = w[e].double(), x[a:b].double()
        out["y"][a:b] = xe @ we.T
        if case["backward"]:
            dye = s["dy"][a:b].double()
            out["dx"][a:b] = dye @ we
            kept = _exact_kept(xe).to(x.dtype).double() if case["kept"] else xe
            out["dw"][e] = dye.T @ kept
    if case["backward"] and not case["experts"]:
        out["dw"] = out["dw"][0]
    return out
