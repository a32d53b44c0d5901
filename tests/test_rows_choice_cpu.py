"""Which kernel a 16-bit product of rows takes and what its workspace holds,
asked of the rule itself (plain C++ without a device), and that the GPU tests
reach every variant."""

import ctypes
import os
import shutil
import subprocess

import pytest

import test_gpu_experts as V

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_expert_grouped_amd", "csrc")
FORWARD, INPUT, WEIGHT = range(3)

SOURCE = """
#include "rows_choice.h"
using namespace mxmoe::rows;
static RowsShape shape(int pass, int64_t rows, int64_t n, int64_t k, int mats, int grouped, int size, int64_t laid_out, int pieces) {
  RowsShape s{};
  s.pass = static_cast<Pass>(pass); s.rows = rows; s.n = n; s.k = k; s.mats = mats; s.grouped = grouped != 0;
  s.out_size = size; s.laid_out = laid_out; s.pieces = pieces != 0;
  return s;
}
extern "C" void choose(int pass, int64_t rows, int64_t n, int64_t k, int mats, int grouped, int size, int64_t laid_out, int pieces,
                       int64_t* out) {
  const RowsShape s = shape(pass, rows, n, k, mats, grouped, size, laid_out, pieces);
  const RowsChoice c = choose_rows(s);
  const int64_t v[] = {c.stream, c.bm, c.slices, c.join, c.wide, c.tiles, least_tiles(s)};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(SOURCE)
    lib = str(d / "choice.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", lib, str(d / "choice.cpp")], check=True)
    fn = ctypes.CDLL(lib).choose
    i, q = ctypes.c_int, ctypes.c_int64
    fn.argtypes = [i, q, q, q, i, i, i, q, i, ctypes.c_void_p]

    def call(which, rows, n, k, mats=0, size=2):
        out = (q * 7)()
        width = n if which == FORWARD else k
        laid = 0
        if which == FORWARD and k % 8:
            laid = (rows + max(1, mats) * n) * k
        fn(which, rows, n, k, max(1, mats), mats > 0, size, laid, width * size % 16 == 0, out)
        return dict(zip(("stream", "bm", "slices", "join", "wide", "tiles", "least"), out))

    return call


def test_the_gpu_cases_reach_every_variant(choose):
    reached = set()
    for rows, mats, n, k in V.SIZES:
        for which in (FORWARD, INPUT, WEIGHT):
            for size in (2, 4) if which == WEIGHT else (2,):
                c = choose(which, rows, n, k, mats, size)
                if c["stream"]:
                    reached.add((which, "stream", 8 if c["tiles"] <= 256 else 4, k % 8 == 0))
                else:
                    reached.add((which, c["bm"], "split" if c["slices"] > 1 else "join" if c["join"] else "wide" if c["wide"] else "odd", size))
    every = {(FORWARD, "stream", w, a) for w in (4, 8) for a in (False, True)}
    every |= {(p, bm, kind, 2) for p in (FORWARD, INPUT) for bm in (64, 128, 256) for kind in ("wide", "odd", "split")}
    every |= {(WEIGHT, bm, kind, 2) for bm in (128, 256) for kind in ("wide", "odd", "split")}
    every |= {(WEIGHT, bm, kind, 4) for bm in (128, 256) for kind in ("wide", "join", "split")}
    assert every - reached == set()
    assert reached - every == set()


def test_the_cases_have_workgroups_with_several_tiles(choose):
    # a stream of steps that runs on over tiles, with half a tile, a whole one and a split last round among them
    for which in (FORWARD, INPUT, WEIGHT):
        for bm in (64, 128, 256):
            if which == WEIGHT and bm == 64:
                continue
            assert any(c["bm"] == bm and not c["stream"] and c["tiles"] > 2 * 256
                       for c in (choose(which, r, n, k, e) for r, e, n, k in V.SIZES)), (which, bm)


def test_what_the_choice_rests_on(choose):
    for which in (FORWARD, INPUT, WEIGHT):
        for rows in (0, 1, 3, 64, 1000, 32768, 1 << 25):
            for n, k in ((1, 1), (8, 65536), (65536, 8), (4096, 7168), (1 << 20, 1), (1 << 20, 1 << 20)):
                for mats in (0, 1, 7, 1024):
                    for size in (2, 4) if which == WEIGHT else (2,):
                        c = choose(which, rows, n, k, mats, size)
                        if c["stream"]:
                            assert which == FORWARD and not c["join"] and c["slices"] == 1
                            continue
                        assert c["bm"] in ((128, 256) if which == WEIGHT else (64, 128, 256))
                        assert c["slices"] in (1, 2, 4, 8, 16, 32, 64)  # (the joining kernel counts on powers of two)
                        assert c["join"] or c["slices"] == 1
                        assert c["wide"] or not c["join"]
                        if size == 4:
                            assert c["wide"]  # (the tile kernel writes fp32 rows in whole pieces only)
                        # slices are for few tiles: with them the count stays far below a launch's limit
                        if c["slices"] > 1:
                            assert c["tiles"] <= c["least"] * c["slices"] and (c["least"] - max(1, mats) * -(-(n if which == FORWARD else k) // 256)) * c["slices"] <= 1 << 20
    # a prompt in tiles of 256 rows, one token straight from memory, long sums of few results in parts
    assert choose(FORWARD, 8192, 4096, 7168)["bm"] == 256 and choose(FORWARD, 1, 4096, 7168)["stream"]
    assert choose(WEIGHT, 32768, 128, 128)["slices"] > 1 and choose(INPUT, 64, 7168, 128)["slices"] > 1
    # operands that are laid out first make the kernel that needs none of it the cheaper one for longer
    last = lambda k: max(r for r in range(1, 2000) if choose(FORWARD, r, 4096, k)["stream"])  # noqa: E731
    assert last(2047) > last(2048)
