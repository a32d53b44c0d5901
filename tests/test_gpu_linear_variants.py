"""The product of MXFP4 matrices in every variant of its kernels, for each type
of result, with several groups of K per wave and several tiles per workgroup;
long rows, and matrices whose offsets pass 32 bits.  The CPU test of the
kernels' choice asks whether CASES reaches every variant."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def uneven(rows, mats):
    """rows shared out over mats matrices: every fifth has none, the others' parts differ by up to four times"""
    part = [0 if i % 5 == 3 else 1 + (7 * i) % 4 for i in range(mats)]
    counts = [rows * p // sum(part) for p in part]
    counts[0] += rows - sum(counts)
    return counts


def ones(rows, mats):
    """one row each for `rows` of mats matrices, far apart"""
    at = {i * mats // rows for i in range(rows)}
    return [int(i in at) for i in range(mats)]


# rows (a number: one matrix, without offsets; a list: rows of each matrix), n, k
STREAM = [
    # a row or a few through eight waves: of 1, 9, 14 and 128 groups of 512, a wave has none, one, two or sixteen
    *[(rows, n, k) for k in (512, 4608, 7168, 65536) for rows, n in ((1, 33), (3, 40), (17, 64))],
    # the same with scales by dwords: 1, 5, 14 and 127 groups, the last of them short
    *[(rows, n, k) for k in (128, 2176, 7040, 64896) for rows, n in ((1, 33), (3, 40), (17, 64))],
    # single scale bytes, units of 16 x 16 and 64 x 32: 1, 4, 9 and 128 groups, the last of them short
    *[(rows, n, k) for k in (96, 2016, 4128, 65504) for rows, n in ((5, 40), (32, 33), (33, 17), (70, 40), (300, 100))],
    (uneven(90, 12), 40, 2016), (uneven(700, 12), 40, 2016), (ones(40, 100), 50, 4128),
    # more units than CUs: four waves, each with up to four groups
    *[(ones(100, 100), 40, k) for k in (512, 2048, 128, 2176)], (1, 8192, 4608), (1, 8190, 7040), (2, 4500, 7168),
    (uneven(150, 30), 56, 640),
]
TILES = [
    # 64 rows, weights read once: a few rows for many matrices; k = 1024 m, 512 m, 128 m, and half a step at the end
    *[(uneven(700, 64), 2048, k) for k in (1024, 2048, 512, 1536, 256, 384, 640)],
    *[(ones(16, 40), 2048, k) for k in (7168, 7680, 7040)],
    # 64 rows, several row tiles for a matrix
    *[(uneven(6000, 100), 520, k) for k in (1024, 2048, 512, 1536, 128, 256, 384, 640)],
    # 64 rows, results that are not whole 16-byte pieces
    *[(uneven(2000, 64), 2049, k) for k in (128, 256, 384, 640, 1024)],
    # 128 rows
    *[(uneven(700, 16), 12000, k) for k in (512, 1536, 128, 256, 384, 640)],
    *[(uneven(4096, 64), 2049, k) for k in (128, 256, 384, 640, 1024)],
    # 256 rows (with fp32 and pieces in part: 128)
    *[(1500, 12000, k) for k in (512, 1536, 128, 256, 384, 640)],
    *[(uneven(9000, 6), 3000, k) for k in (512, 384)],
    *[(8192, 2049, k) for k in (128, 256, 384, 640, 1024)],
]
CASES = STREAM + TILES


def counts_of(rows):
    return rows if isinstance(rows, list) else [rows]


def name_of(rows, n, k):
    return f"{rows}x{n}x{k}" if isinstance(rows, int) else f"{sum(rows)}of{len(rows)}x{n}x{k}"


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


def random_mx4(shape, k, g, lo=120, hi=131):
    """codes of every value, scales 2^-7 .. 2^3"""
    r = lambda a, b, n: torch.randint(a, b, (*shape, n), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return r(0, 256, k // 2), r(lo, hi, k // 32)


def values(codes, scales):
    """the values of a canonical MXFP4 matrix, float64"""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).reshape(codes.shape[0], -1, 32)
    return (v * torch.exp2(scales.double() - 127)[:, :, None]).reshape(codes.shape[0], -1)


def assert_product(got, a, w, k, dtype):
    # products of two E2M1 values and powers of two are exact; adding k of them in fp32, in any order, is off by at
    # most k 2^-24 of the sum of magnitudes, and the result is rounded once (2^-25: fp16's smallest numbers)
    ref, mag = a @ w.T, a.abs() @ w.abs().T
    bound = k * 2.0 ** -24 * mag
    bound += torch.finfo(DT[dtype]).eps / 2 * (ref.abs() + bound) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert bool(((got.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,n,k", CASES, ids=[name_of(*c) for c in CASES])
def test_every_variant(L, rows, n, k, dtype):
    counts = counts_of(rows)
    g = torch.Generator(device="cuda").manual_seed(n + k + sum(counts))
    ac, asc = random_mx4((sum(counts),), k, g)
    wc, wsc = random_mx4((len(counts), n), k, g)
    if dtype == "fp16":
        asc -= 9  # sums within fp16's range
    if isinstance(rows, list):
        offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        y = L.linear_mx4(ac, asc, wc, wsc, offsets=offsets, dtype=DT[dtype])
    else:
        y = L.linear_mx4(ac, asc, wc[0], wsc[0], dtype=DT[dtype])
    at = 0
    for e, c in enumerate(counts):
        if c:
            assert_product(y[at:at + c], values(ac[at:at + c], asc[at:at + c]), values(wc[e], wsc[e]), k, dtype)
        at += c


@pytest.mark.parametrize("rows,n,k", [(40, 56, 96), (600, 2056, 2016), (2048, 4096, 2880)])
def test_zero_blocks_at_the_end_of_k_add_nothing(L, rows, n, k):
    # a k that tiles do not take, padded to one that they take: held to the bound of the sum without the padding
    g = torch.Generator(device="cuda").manual_seed(k)
    ac, asc = random_mx4((rows,), k, g)
    wc, wsc = random_mx4((n,), k, g)
    more = -k % 128
    pad = torch.nn.functional.pad
    y = L.linear_mx4(pad(ac, (0, more // 2)), pad(asc, (0, more // 32)), pad(wc, (0, more // 2)), pad(wsc, (0, more // 32)),
                     dtype=torch.float32)
    assert_product(y, values(ac, asc), values(wc, wsc), k, "fp32")


@pytest.mark.parametrize("rows,n,k", [(3, 40, 512), (70, 40, 96), (600, 8192, 512), (600, 8191, 384)])
@pytest.mark.parametrize("ld", [(1 << 22) - 8, 1 << 22, (1 << 22) + 8])
def test_rows_of_y_far_apart(L, rows, n, k, ld):
    # 256 rows of y below, at and above the 2^31 bytes that a tile's stores reach; the last rows lie past 2^32 bytes
    g = torch.Generator(device="cuda").manual_seed(n + k)
    ac, asc = random_mx4((rows,), k, g)
    wc, wsc = random_mx4((n,), k, g)
    asc -= 9
    whole = torch.full((rows * ld,), 7.0, dtype=torch.float16, device="cuda")
    out = whole.view(rows, ld)[:, :n]
    L.linear_mx4(ac, asc, wc, wsc, out=out)
    assert_product(out, values(ac, asc), values(wc, wsc), k, "fp16")
    out.fill_(7.0)
    for part in whole.split(1 << 30):
        assert bool((part == 7).all())


def check_some_rows(y, ac, asc, wc, wsc, k, dtype):
    """the first and the last rows, and some between"""
    n = y.shape[0]
    pick = torch.cat([torch.arange(64), torch.arange(n // 2, n // 2 + 64), torch.arange(n - 64, n)]).cuda()
    assert_product(y[pick], values(ac[pick], asc[pick]), values(wc, wsc), k, dtype)


@pytest.mark.parametrize("rows,n,k", [((1 << 18) + 5, 40, 16384 + 512), ((1 << 18) + 5, 40, 16384 + 96), ((1 << 18) + 5, 8200, 128)])
def test_rows_past_32_bits(L, rows, n, k):
    # more than 2^31 bytes of codes, or elements of y
    g = torch.Generator(device="cuda").manual_seed(k)
    ac, asc = random_mx4((rows,), k, g)
    wc, wsc = random_mx4((n,), k, g)
    check_some_rows(L.linear_mx4(ac, asc, wc, wsc), ac, asc, wc, wsc, k, "bf16")


@pytest.mark.parametrize("per", [1, 70])
def test_matrices_past_32_bits(L, per):
    # more than 2^32 bytes of weights, a few rows and row tiles for the first and the last matrices
    mats, n, k = 600, 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(per)
    wc, wsc = random_mx4((mats, n), k, g)
    counts = [per * (e < 3 or e >= mats - 3) for e in range(mats)]
    ac, asc = random_mx4((sum(counts),), k, g)
    y = L.linear_mx4(ac, asc, wc, wsc, offsets=torch.tensor([0] + counts, device="cuda").cumsum(0).int(), dtype=torch.float32)
    at = 0
    for e, c in enumerate(counts):
        if c:
            assert_product(y[at:at + c], values(ac[at:at + c], asc[at:at + c]), values(wc[e], wsc[e]), k, "fp32")
        at += c
