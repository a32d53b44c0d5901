"""What the exact products of the GPU tests reach and see, on the CPU: the real
tiles of each of their calls, counted from its offsets and the rule's choice,
and that a sum with products left out does not pass for the whole one."""

import pytest
import torch

import test_gpu_experts as V
import test_gpu_experts_exact as E
from test_rows_choice_cpu import FORWARD, INPUT, WEIGHT, choose  # noqa: F401

CUS = 256


def tiles_of(which, n, k, cuts, c):
    """-> (tiles in all, workgroups, rows of the tiles that two workgroups share in the last round)"""
    ntn, bm = -(-(n if which == FORWARD else k) // 256), c["bm"]
    lens = [n if which == WEIGHT else b - a for a, b in zip(cuts, cuts[1:])]
    row_tiles = [-(-r // bm) for r in lens]
    per_slice = sum(row_tiles) * ntn
    tiles, grid = per_slice * c["slices"], max(1, min(c["tiles"], CUS))
    rest, shared = tiles % grid, []
    if which != WEIGHT and bm == 256 and 2 * rest <= grid:
        for at in range(tiles - rest, tiles):
            at, e = at % per_slice, 0
            while at >= row_tiles[e] * ntn:
                at -= row_tiles[e] * ntn
                e += 1
            panel, within = divmod(at, 4 * ntn)  # four row tiles, column block by column block
            tile = 4 * panel + within % min(4, row_tiles[e] - 4 * panel)
            shared.append(min(256, lens[e] - 256 * tile))
    return tiles, grid, shared


def store_of(c):
    return "parts" if c["slices"] > 1 else "join" if c["join"] else "wide" if c["wide"] else "odd"


def test_every_kind_of_tile_follows_another_in_its_workgroup(choose):
    several, shared = set(), set()
    for rows, mats, n, k in E.SIZES:
        for which in (FORWARD, INPUT, WEIGHT):
            for size in (2, 4) if which == WEIGHT else (2,):
                c = choose(which, rows, n, k, mats, size)
                if c["stream"]:
                    continue
                for kind in E.KINDS if mats else E.KINDS[:1]:
                    tiles, grid, parts = tiles_of(which, n, k, E.cuts_of(rows, mats, kind, k), c)
                    if tiles > grid:
                        several.add((which, c["bm"], store_of(c), size))
                    if tiles > grid and max(parts, default=0) > 128:
                        shared.add((which, store_of(c)))
    every = {(p, bm, kind, 2) for p in (FORWARD, INPUT) for bm in (64, 128, 256) for kind in ("wide", "odd", "parts")}
    every |= {(WEIGHT, bm, kind, 2) for bm in (128, 256) for kind in ("wide", "odd")}
    every |= {(WEIGHT, bm, kind, 4) for bm in (128, 256) for kind in ("wide", "join")}
    assert every - several == set()
    # the second of two workgroups has rows of its own
    assert {(p, kind) for p in (FORWARD, INPUT) for kind in ("wide", "odd", "parts")} - shared == set()


def test_some_tiles_are_of_several_steps(choose):
    # more than the ring has slots (two or three): at least four steps of 64
    for which in (FORWARD, INPUT, WEIGHT):
        for bm in (128, 256) if which == WEIGHT else (64, 128, 256):
            for store in ("wide", "odd"):
                assert any(c["bm"] == bm and store_of(c) == store and not c["stream"] and length >= 256 and c["tiles"] > CUS
                           for r, e, n, k in E.SIZES for c in (choose(which, r, n, k, e),)
                           for length in ([k, n, r // max(1, e)][which],)), (which, bm, store)


@pytest.mark.parametrize("rows,mats,n,k", [(22940, 0, 1336, 34), (36297, 0, 258, 263), (31257, 20, 400, 52), (5608, 20, 24, 3109)])
def test_a_sum_with_rows_left_out_is_another(rows, mats, n, k):
    assert (rows, mats, n, k) in E.SIZES
    x, w, dy = E.operands(rows, mats, n, k)
    cuts = E.cuts_of(rows, mats, "even", k)
    a, b = cuts[0], cuts[1]
    whole = dy[a:b].T @ x[a:b]
    assert float((dy[a:b].abs().T @ x[a:b].abs()).max()) < 2 ** 24
    last = a + (b - a) // 64 * 64 if (b - a) % 64 else b
    for without in (slice(last, b), slice(last - 64, last), slice(a, a + 64), slice(b - 1, b), slice((a + b) // 2, (a + b) // 2 + 1)):
        if without.start == without.stop:
            continue
        missing = dy[without].T @ x[without]
        for dt in (torch.bfloat16, torch.float16, torch.float32):
            assert not torch.equal((whole - missing).to(dt), whole.to(dt)), (without, dt)
            with pytest.raises(AssertionError, match="differ"):
                E.equal((whole - missing).to(dt), whole)


def test_rows_left_out_of_300000_are_seen():
    # the sums of the largest call, for a few of its columns: the rows past 2^32 bytes of x, a last step, one row
    rows, row_bytes = 300012, 2 * 4160
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randint(-1, 2, (rows, c), generator=g, dtype=torch.int8).double() for c in (32, 16))
    whole = dy.T @ x
    first = 299999  # (of the second matrix)
    past = -(-(1 << 32) // row_bytes) - first
    for without in (slice(past, rows), slice(rows - rows % 64, rows), slice(rows - 1, rows)):
        missing = dy[without].T @ x[without]
        with pytest.raises(AssertionError, match="differ"):
            E.equal((whole - missing).float(), whole)
