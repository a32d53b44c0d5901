"""The MXFP4 quantiser, its inverse and the product of two MXFP4 matrices on
the GPU, against the oracle's formats (float64)."""

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
def L():
    from mxfp4_expert_grouped_amd import layer
    return layer


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def assert_quantized(L, x):
    """codes and scales equal to the oracle's, byte for byte"""
    codes, scales = L.quantize_mx4(x)
    rc, rs = X.mx_quantize(f64(x), "e2m1")
    assert codes.shape == (x.shape[0], x.shape[1] // 2) and scales.shape == (x.shape[0], x.shape[1] // 32)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    return codes, scales


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (7, 1056), (33, 2048), (130, 64), (1025, 32)])
def test_quantize_matches_oracle(L, dtype, rows, cols):
    g = torch.Generator().manual_seed(rows * 7919 + cols)
    x = torch.randn((rows, cols), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g))
    assert_quantized(L, x.clamp(-60000, 60000).to(DT[dtype]).cuda())


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_midpoints_signs_and_saturation(L, dtype):
    # every midpoint of the grid and its neighbours, both signs, with amax in [4, 8): 2^0 is the scale
    mids = [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0]
    vals = []
    eps = 2.0 ** -6
    for m in mids:
        vals += [m, m * (1 - eps), m * (1 + eps)]
    vals += [7.9375]
    vals = [v for v in vals if v < 8]
    rows = []
    for v in vals:
        for s in (1.0, -1.0):
            r = [4.0, -0.0, 0.0] + [s * v] * 29
            rows.append(r)
    x = torch.tensor(rows, dtype=torch.float64)
    for e in (0, -9, 11):
        assert_quantized(L, (x * 2.0 ** e).to(DT[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_extreme_exponents(L, dtype):
    # block maxima from the subnormal numbers (scale clamped at 2^-127) to the largest finite one
    g = torch.Generator().manual_seed(5)
    m = 1 + torch.rand((300, 32), generator=g, dtype=torch.float64)
    m = m * torch.where(torch.rand((300, 32), generator=g) < 0.5, -1.0, 1.0)
    e = torch.cat([torch.arange(-149, -100), torch.linspace(-100, 110, 230).round(), torch.arange(107, 128)])[:, None]
    fall = torch.randint(0, 6, (300, 32), generator=g)
    x = (m * torch.exp2(e.double() - fall)).to(torch.float32)
    x = torch.where(torch.isinf(x), torch.full_like(x, 3.0e38), x).to(DT[dtype])
    x = torch.where(torch.isinf(x), torch.full_like(x, 3.0e38), x)
    assert torch.isfinite(x).all()
    codes, scales = assert_quantized(L, x.cuda())
    for out in ("bf16", "fp32"):
        v = L.dequantize_mx4(codes, scales, DT[out])
        ref = X.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), "e2m1")
        assert np.array_equal(f64(v), ref)


def test_quantize_subnormal_halves(L):
    x = (torch.arange(-64, 64, dtype=torch.float64) * 2.0 ** -24).reshape(4, 32).to(torch.float16)
    codes, scales = assert_quantized(L, x.cuda())
    ref = X.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), "e2m1")
    assert np.array_equal(f64(L.dequantize_mx4(codes, scales, torch.float16)), ref)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantize_poisons_a_block_that_is_not_finite(L, dtype, bad):
    g = torch.Generator().manual_seed(11)
    x = torch.randn((3, 128), generator=g)
    x[1, 70] = bad
    x = x.to(DT[dtype])
    codes, scales = L.quantize_mx4(x.cuda())
    good = x.clone()
    good[1, 64:96] = 0
    rc, rs = X.mx_quantize(f64(good), "e2m1")
    rs[1, 2] = 255
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    v = f64(L.dequantize_mx4(codes, scales, DT[dtype]))
    assert np.isnan(v[1, 64:96]).all() and np.isfinite(np.delete(v.ravel(), np.arange(128 + 64, 128 + 96))).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_strided_and_unaligned_rows(L, dtype):
    g = torch.Generator().manual_seed(12)
    base = torch.randn((9, 200), generator=g).to(DT[dtype]).cuda()
    for x in (base[:, 8:104], base[:, 1:97], base[::2, 3:163], base[:1, 5:69], base[2:3].expand(4, -1)[:, :64],
              torch.randn((64, 10), generator=g).to(DT[dtype]).cuda().t()):
        assert_quantized(L, x)


def test_quantize_empty(L):
    for shape in ((0, 64), (5, 0)):
        c, s = L.quantize_mx4(torch.empty(shape, device="cuda"))
        assert c.shape == (shape[0], shape[1] // 2) and s.shape == (shape[0], shape[1] // 32)
        assert L.dequantize_mx4(c, s).shape == shape


@pytest.mark.parametrize("dtype", list(DT))
def test_dequantize_every_code_and_scale(L, dtype):
    # each scale byte with all 16 codes twice; rounded once to the type
    codes = torch.from_numpy(X.pack_fp4(np.tile(np.arange(16, dtype=np.uint8), (256, 2)))).cuda()
    scales = torch.arange(256, dtype=torch.uint8).reshape(256, 1).cuda()
    v = L.dequantize_mx4(codes, scales, DT[dtype])
    exact = torch.from_numpy(X.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), "e2m1"))
    ref = exact.to(torch.float32).to(DT[dtype])  # the fp32 step is exact or overflows to the same infinity
    assert torch.equal(v.cpu().isnan(), ref.isnan())
    assert torch.equal(v.cpu().nan_to_num(7.0), ref.nan_to_num(7.0))
    assert torch.equal(torch.signbit(v.cpu()[:255]), torch.signbit(ref[:255]))


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------


def random_mx4(shape, k, seed, lo=120, hi=131):
    """random codes of every value and scales 2^-7 .. 2^3 (the sums then need more bits than fp32 has)"""
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (*shape, k // 2), dtype=np.uint8),
            rng.integers(lo, hi, (*shape, k // 32), dtype=np.uint8))


def linear_ref(ac, asc, wc, wsc, offsets):
    """y and the sum of the terms' magnitudes, float64"""
    a = X.mx_decode(ac, asc, "e2m1")
    rows, n = a.shape[0], wc.shape[-2]
    y, mag = np.zeros((rows, n)), np.zeros((rows, n))
    for e in range(wc.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            w = X.mx_decode(wc[e], wsc[e], "e2m1")
            y[lo:hi] = a[lo:hi] @ w.T
            mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w).T
    return y, mag


def assert_linear(got, y, mag, k, dtype):
    # every product of two E2M1 values and powers of two is exact; adding k of
    # them in fp32 in any order is off by at most k half steps of partial sums,
    # each at most the sum of magnitudes: k 2^-24 mag.  The result is rounded
    # once: half a step of the type, eps/2 relative, and 2^-25 for fp16's
    # smallest numbers
    got = f64(got)
    half = torch.finfo(DT[dtype]).eps / 2
    bound = k * 2.0 ** -24 * mag
    bound += half * (np.abs(y) + bound) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    bad = ~(np.abs(got - y) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], y[bad][:5])


def run_linear(L, ac, asc, wc, wsc, offsets, dtype, grouped=True):
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    if grouped:
        return L.linear_mx4(c(ac), c(asc), c(wc), c(wsc), offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                            dtype=DT[dtype])
    return L.linear_mx4(c(ac), c(asc), c(wc[0]), c(wsc[0]), dtype=DT[dtype])


KS = [32, 96, 128, 160, 384, 512, 640, 1024, 1536, 2048]


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("rows,n,dtype", [(1, 1, "fp32"), (1, 130, "bf16"), (5, 64, "fp16"), (16, 17, "fp32"),
                                          (33, 256, "bf16"), (70, 300, "fp32"), (200, 129, "bf16"), (300, 600, "fp32")])
def test_linear_one_matrix(L, k, rows, n, dtype):
    ac, asc = random_mx4((rows,), k, 100 + k + rows)
    wc, wsc = random_mx4((1, n), k, 200 + k + n)
    if dtype == "fp16":
        asc -= 6  # sums within fp16's range
    y, mag = linear_ref(ac, asc, wc, wsc, [0, rows])
    assert_linear(run_linear(L, ac, asc, wc, wsc, None, dtype, grouped=False), y, mag, k, dtype)


@pytest.mark.parametrize("k", [96, 128, 512, 640, 1024])
@pytest.mark.parametrize("counts,n,dtype", [
    ([1], 64, "bf16"), ([0, 1, 0, 0, 3], 100, "fp32"), ([16, 17, 0, 15, 1, 33], 48, "bf16"),
    ([40, 0, 64, 65, 1, 90], 260, "fp32"), ([300, 1, 0, 257, 256, 255], 272, "bf16"), ([0, 0, 1000, 2], 520, "fp32"),
    ([1] * 70, 32, "bf16"),
])
def test_linear_by_experts(L, k, counts, n, dtype):
    offsets = [0] + np.cumsum(counts).tolist()
    rows = offsets[-1]
    ac, asc = random_mx4((rows,), k, 300 + k + rows)
    wc, wsc = random_mx4((len(counts), n), k, 400 + k + n)
    y, mag = linear_ref(ac, asc, wc, wsc, offsets)
    assert_linear(run_linear(L, ac, asc, wc, wsc, offsets, dtype), y, mag, k, dtype)


# enough products for tiles of 64, 128 and 256 rows, whole and ragged ones; widths that are whole 16-byte pieces
# of y, or not; every way in which the scales come (k a multiple of 1024, 512, 256, 128) with few and several steps
@pytest.mark.parametrize("k", [128, 256, 384, 512, 640, 1024, 1536, 2048])
@pytest.mark.parametrize("rows,n,dtype", [(500, 8192, "bf16"), (300, 8184, "fp32"), (1001, 8192, "bf16"), (1024, 8190, "fp16"),
                                          (2000, 8184, "bf16"), (2048, 8192, "fp32"), (2047, 8191, "bf16"), (33, 12000, "fp32")])
def test_linear_in_tiles(L, k, rows, n, dtype):
    ac, asc = random_mx4((rows,), k, 500 + k + rows)
    wc, wsc = random_mx4((1, n), k, 600 + k + n)
    if dtype == "fp16":
        asc -= 6
    y, mag = linear_ref(ac, asc, wc, wsc, [0, rows])
    assert_linear(run_linear(L, ac, asc, wc, wsc, None, dtype, grouped=False), y, mag, k, dtype)


@pytest.mark.parametrize("k", [128, 384, 512, 1024, 1536])
@pytest.mark.parametrize("counts,n,dtype", [
    ([0, 300, 17, 64, 65, 128, 129, 1, 255, 256, 257, 0, 90, 33, 500, 63], 2304, "bf16"),
    ([1, 0, 2, 64, 1] * 13, 2048, "fp32"), ([40] * 40 + [0] * 20, 1544, "fp16"), ([700, 0, 0, 900], 4088, "fp32"),
])
def test_linear_by_experts_in_tiles(L, k, counts, n, dtype):
    offsets = [0] + np.cumsum(counts).tolist()
    ac, asc = random_mx4((offsets[-1],), k, 700 + k + n)
    wc, wsc = random_mx4((len(counts), n), k, 800 + k + n)
    if dtype == "fp16":
        asc -= 6
    y, mag = linear_ref(ac, asc, wc, wsc, offsets)
    assert_linear(run_linear(L, ac, asc, wc, wsc, offsets, dtype), y, mag, k, dtype)


@pytest.mark.parametrize("k,n,per", [(512, 64, 2), (512, 200, 40), (512, 300, 200), (96, 40, 20), (512, 8192, 100),
                                     (384, 8191, 400), (96, 300, 100)])
def test_linear_leaves_rows_outside_the_offsets(L, k, n, per):
    # rows before the first offset and behind the last stay as they were, and a strided out keeps its gaps
    counts = [per, 0, per + 3]
    offsets = [3] + (3 + np.cumsum(counts)).tolist()
    rows = offsets[-1] + 37
    ac, asc = random_mx4((rows,), k, 21)
    wc, wsc = random_mx4((3, n), k, 22)
    asc[:3] = 255  # poison that nothing reads
    asc[offsets[-1]:] = 255
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    whole = torch.full((rows, n + 5), 7.25, device="cuda")
    out = whole[:, 2:2 + n]
    L.linear_mx4(c(ac), c(asc), c(wc), c(wsc), offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    y, mag = linear_ref(np.where(asc[:, :1] == 255, 0, ac).astype(np.uint8), np.where(asc == 255, 127, asc).astype(np.uint8), wc, wsc, offsets)
    lo, hi = offsets[0], offsets[-1]
    assert_linear(out[lo:hi], y[lo:hi], mag[lo:hi], k, "fp32")
    whole[lo:hi, 2:2 + n] = 7.25
    assert (whole == 7.25).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,gap", [(4089, 0), (4090, 3), (4091, 1), (4092, 0), (4093, 5), (4094, 1), (4095, 8), (4096, 1)])
def test_linear_rows_of_y_anywhere(L, n, gap, dtype):
    # every number of columns in a row's last piece, rows that begin anywhere, in tiles of many rows: what lies
    # between the rows, before the first and behind the last, stays as it was
    k, offsets = 256, [0, 1200, 1200, 1777, 2048]
    ac, asc = random_mx4((2048,), k, 900 + n)
    wc, wsc = random_mx4((4, n), k, 1000 + n)
    if dtype == "fp16":
        asc -= 6
    y, mag = linear_ref(ac, asc, wc, wsc, offsets)
    ld, lead = n + gap, 1
    flat = torch.full((lead + 2048 * ld + 64,), 7.0, dtype=DT[dtype], device="cuda")
    out = flat[lead:lead + 2048 * ld].view(2048, ld)[:, :n]
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    L.linear_mx4(c(ac), c(asc), c(wc), c(wsc), offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    assert_linear(out, y, mag, k, dtype)
    assert bool((flat[:lead] == 7).all()) and bool((flat[lead + 2048 * ld:] == 7).all())
    assert bool((flat[lead:lead + 2048 * ld].view(2048, ld)[:, n:] == 7).all())


@pytest.mark.parametrize("rows,k", [(4, 512), (100, 512), (4, 96), (600, 1024), (3000, 640)])
def test_linear_offsets_out_of_range_stay_inside(L, rows, k):
    n = 40 if rows < 3000 else 2000
    ac, asc = random_mx4((rows,), k, 31)
    wc, wsc = random_mx4((4, n), k, 32)
    guard = torch.full((rows + 64, n), 3.5, device="cuda")
    offsets = torch.tensor([-50, 2, 1, 10 ** 9, -7], dtype=torch.int32, device="cuda")
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    L.linear_mx4(c(ac), c(asc), c(wc), c(wsc), offsets=offsets, out=guard[:rows])
    # matrix 0: rows 0-1; matrix 1: none (its end lies before its start); matrix 2: rows 1 .. rows; matrix 3: none
    y0, m0 = linear_ref(ac, asc, wc, wsc, [0, 2, 2, 2, 2])
    y2, m2 = linear_ref(ac, asc, wc, wsc, [1, 1, 1, rows, rows])
    assert_linear(guard[:1], y0[:1], m0[:1], k, "fp32")
    assert_linear(guard[2:rows], y2[2:], m2[2:], k, "fp32")  # row 1 is in both ranges: either
    assert (guard[rows:] == 3.5).all()


@pytest.mark.parametrize("rows,k,n", [(3, 512, 40), (80, 512, 300), (300, 1024, 300), (3, 96, 40), (300, 128, 260),
                                      (600, 1024, 8192), (2048, 384, 8192)])
def test_linear_nan_scales(L, rows, k, n):
    # a NaN block of a row poisons that row alone, one of a weight row that column alone
    ac, asc = random_mx4((rows,), k, 41)
    wc, wsc = random_mx4((1, n), k, 42)
    y, mag = linear_ref(ac, asc, wc, wsc, [0, rows])
    asc[1, k // 32 - 1] = 255
    wsc[0, n - 2, 0] = 255
    got = run_linear(L, ac, asc, wc, wsc, None, "fp32", grouped=False)
    nan = np.zeros((rows, n), dtype=bool)
    nan[1] = True
    nan[:, n - 2] = True
    assert np.array_equal(np.isnan(f64(got)), nan)
    assert_linear(got.nan_to_num(0.0), np.where(nan, 0, y), mag, k, "fp32")


@pytest.mark.parametrize("rows,k,n", [(4, 512, 40), (90, 96, 64), (700, 1024, 4096), (2048, 384, 8192)])
def test_linear_of_a_row_that_is_not_finite(L, rows, k, n):
    # what the quantiser makes of an infinity (scale 255, codes 0) poisons the row's results, and no other's
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((rows, k), generator=g, device="cuda")
    w = torch.randn((n, k), generator=g, device="cuda")
    wc, ws = L.quantize_mx4(w)
    c, s = L.quantize_mx4(x)
    good = L.linear_mx4(c, s, wc, ws)
    x[2, k - 5] = float("inf")
    c, s = L.quantize_mx4(x)
    got = L.linear_mx4(c, s, wc, ws)
    assert got[2].isnan().all()
    got[2] = good[2]
    assert torch.equal(got, good)


@pytest.mark.parametrize("rows,k,n", [(2, 512, 20), (40, 512, 256), (300, 512, 256), (2, 128, 20), (600, 512, 8192),
                                      (600, 96, 300)])
def test_linear_extreme_scales(L, rows, k, n):
    # 2^-127 and large scales meet: products inside fp32's range are right
    ac, asc = random_mx4((rows,), k, 51)
    wc, wsc = random_mx4((1, n), k, 52)
    asc[:] = 0
    wsc[:] = 250
    y, mag = linear_ref(ac, asc, wc, wsc, [0, rows])
    assert_linear(run_linear(L, ac, asc, wc, wsc, None, "fp32", grouped=False), y, mag, k, "fp32")


def test_linear_of_slices_and_copies(L):
    # weights of one expert sliced out of the stack, rows sliced out of a larger matrix: unaligned views are copied
    k, n, rows = 160, 33, 9
    ac, asc = random_mx4((rows + 1,), k, 61)
    wc, wsc = random_mx4((3, n), k, 62)
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    got = L.linear_mx4(c(ac)[1:], c(asc)[1:], c(wc)[2], c(wsc)[2], dtype=torch.float32)
    y, mag = linear_ref(ac[1:], asc[1:], wc[2:], wsc[2:], [0, rows])
    assert_linear(got, y, mag, k, "fp32")
    got = L.linear_mx4(c(ac)[1:], c(asc)[1:], c(wc).flip(0)[0], c(wsc).flip(0)[0], dtype=torch.float32)
    assert_linear(got, y, mag, k, "fp32")


@pytest.mark.parametrize("rows,n", [(20, 40), (700, 4096)])
def test_linear_unaligned_scales(L, rows, n):
    # scale bytes that start one byte off: the loads go by the alignment
    k = 1024
    ac, asc = random_mx4((rows,), k, 63)
    wc, wsc = random_mx4((1, n), k, 64)
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    y, mag = linear_ref(ac, asc, wc, wsc, [0, rows])
    for off in (1, 4):
        a_s = torch.empty(asc.size + off, dtype=torch.uint8, device="cuda")[off:].view(asc.shape)
        w_s = torch.empty(wsc.size + off, dtype=torch.uint8, device="cuda")[off:].view(wsc[0].shape)
        a_s.copy_(c(asc))
        w_s.copy_(c(wsc[0]))
        assert_linear(L.linear_mx4(c(ac), a_s, c(wc[0]), w_s, dtype=torch.float32), y, mag, k, "fp32")


def test_linear_empty(L):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    assert L.linear_mx4(z(0, 64), z(0, 4), z(8, 64), z(8, 4)).shape == (0, 8)
    assert L.linear_mx4(z(3, 64), z(3, 4), z(0, 64), z(0, 4)).shape == (3, 0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full((3, 8), 2.5, device="cuda")
    L.linear_mx4(z(3, 64), z(3, 4), z(2, 8, 64), z(2, 8, 4), offsets=off, out=out)
    assert (out == 2.5).all()


@pytest.mark.parametrize("rows,n,k,mats", [(1, 256, 1024, 1), (64, 300, 1024, 3), (700, 512, 2048, 2), (900, 4096, 1024, 3),
                                           (2500, 8192, 512, 2)])
def test_quantize_and_linear_in_a_replayed_graph(L, rows, n, k, mats):
    # captured once, replayed with new inputs between eager calls of the same
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((rows, k), generator=g, device="cuda").bfloat16()
    w = [L.quantize_mx4(torch.randn((n, k), generator=g, device="cuda")) for _ in range(mats)]
    wc, ws = torch.stack([c for c, _ in w]), torch.stack([s for _, s in w])
    offsets = torch.linspace(0, rows, mats + 1).int().cuda()

    def call():
        c, s = L.quantize_mx4(x)
        return L.linear_mx4(c, s, wc, ws, offsets=offsets)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    for i in range(4):
        x.copy_(torch.randn((rows, k), generator=g, device="cuda"))
        offsets[1:mats] = torch.randint(0, rows + 1, (mats - 1,), generator=g, device="cuda").sort()[0].int()
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, call())


@pytest.mark.parametrize("rows", [2, 40, 600, 2100])
def test_linear_on_two_streams(L, rows):
    k, n = 1024, 512 if rows < 600 else 8192
    c = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    sets = []
    for i in range(2):
        ac, asc = random_mx4((rows,), k, 71 + i)
        wc, wsc = random_mx4((1, n), k, 81 + i)
        sets.append((c(ac), c(asc), c(wc[0]), c(wsc[0])))
    ref = [L.linear_mx4(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(L.linear_mx4(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, ref[i])


def test_refusals(L):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        L.quantize_mx4(torch.zeros(4, 48, device="cuda"))
    with pytest.raises(ValueError):
        L.quantize_mx4(torch.zeros(64, device="cuda"))
    with pytest.raises(ValueError):
        L.quantize_mx4(torch.zeros(4, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        L.quantize_mx4(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        L.dequantize_mx4(z(4, 16), z(4, 2))
    with pytest.raises(ValueError):
        L.linear_mx4(z(4, 64), z(4, 4), z(8, 32), z(8, 2))
    with pytest.raises(ValueError):
        L.linear_mx4(z(4, 64), z(4, 4), z(2, 8, 64), z(2, 8, 4))
    with pytest.raises(ValueError):
        L.linear_mx4(z(4, 64), z(4, 4), z(2, 8, 64), z(2, 8, 4), offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        L.linear_mx4(z(4, 64), z(4, 4), z(2, 8, 64), z(2, 8, 4), offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        L.linear_mx4(z(4, 64), z(4, 4), z(8, 64), z(8, 4), out=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        L.linear_mx4(z(4, 64), z(4, 4), z(8, 64), z(8, 4), dtype=torch.float64)
