"""Which kernel a product of MXFP4 matrices takes, asked of the rule itself
(plain C++ without a device), and that the GPU tests reach every one."""

import ctypes
import os
import shutil
import subprocess
from collections import Counter

import pytest

import test_gpu_linear_variants as V

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_expert_grouped_amd", "csrc")
CUS = 256

SOURCE = """
#include "linear_choice.h"
extern "C" void choose(int64_t rows, int64_t n, int64_t k, int mats, int grouped, int size, int64_t row_bytes, int pieces,
                       int scale_align, int cus, int64_t* out) {
  const mxmoe::LinearShape s{rows, n, k, mats, grouped != 0, size, row_bytes, pieces != 0, scale_align, cus};
  const mxmoe::LinearChoice c = mxmoe::choose_linear(s);
  const int64_t v[] = {c.bm, c.scales, c.wide, c.once, c.mt, c.nb, c.waves};
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
    fn.argtypes = [q, q, q, i, i, i, q, i, i, i, ctypes.c_void_p]

    def call(rows, n, k, mats=1, grouped=False, size=2, gap=0, scale_align=None):
        # a tensor's scales begin on 16 bytes: what their rows begin on is k's doing
        align = scale_align or (16 if k % 512 == 0 else 4 if k % 128 == 0 else 1)
        ld = (n + gap) * size
        out = (q * 7)()
        fn(rows, n, k, mats, grouped, size, ld, ld % 16 == 0 and n * size % 16 == 0, align, CUS, out)
        return tuple(out)

    return call


def test_the_gpu_cases_reach_every_variant(choose):
    # (type, variant): those that are built; tiles in which a workgroup had more than one are counted apart
    reached, again = Counter(), Counter()
    for rows, n, k in V.CASES:
        counts = V.counts_of(rows)
        for name, dtype in V.DT.items():
            v = choose(sum(counts), n, k, len(counts), isinstance(rows, list), dtype.itemsize)
            reached[name, v] += 1
            if v[0] and sum(-(-c // v[0]) for c in counts) * -(-n // 256) > CUS:
                again[name, v] += 1
    stream = [(0, 0, 0, 0, 1, 1, 8), (0, 0, 0, 0, 1, 1, 4), (0, 1, 0, 0, 1, 1, 8), (0, 1, 0, 0, 1, 1, 4), (0, 2, 0, 0, 1, 1, 4),
              (0, 2, 0, 0, 4, 2, 8)]
    tile = [(64, gs, 1, once, 0, 0, 0) for gs in (0, 2, 4) for once in (0, 1)]
    tile += [(bm, gs, 1, 0, 0, 0, 0) for bm in (128, 256) for gs in (0, 2)]
    tile += [(bm, 0, 0, 0, 0, 0, 0) for bm in (64, 128, 256)]
    every = {(t, v) for t in V.DT for v in stream + tile} - {("fp32", (256, 0, 0, 0, 0, 0, 0))}
    assert set(reached) == every
    assert set(again) == {(t, v) for t, v in every if v[0]}


def test_the_streaming_cases_have_waves_without_one_with_one_and_with_several_groups(choose):
    groups = {}
    for rows, n, k in V.STREAM:
        counts = V.counts_of(rows)
        v = choose(sum(counts), n, k, len(counts), isinstance(rows, list))
        if v[0]:
            continue
        q, waves = -(-k // 512), v[6]
        groups.setdefault(v, set()).update({q // waves, -(-q // waves)})
    for v, of in groups.items():
        assert {0, 1, 2} <= of, (v, of)


def test_what_the_choice_rests_on(choose):
    assert choose(8192, 4096, 7168)[0] == 256 and choose(1, 4096, 7168)[0] == 0
    # a k that tiles do not take, scales on no 4 bytes, rows of y too far apart for a tile's stores
    assert choose(8192, 4096, 2016)[0] == 0 and choose(8192, 4096, 7168, scale_align=1)[0] == 0
    at_limit = (1 << 22) - 4096
    assert choose(8192, 4096, 7168, gap=at_limit)[0] == 256 and choose(8192, 4096, 7168, gap=at_limit + 1)[0] == 0
    # scales on 4 bytes only: by dwords
    assert choose(8192, 4096, 7168, scale_align=4)[1] == 0
    assert choose(8192, 4095, 7168)[2] == 0 and choose(8192, 4096, 7168, gap=1)[2] == 0
