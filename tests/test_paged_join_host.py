"""The join's way from the CTA numbers in the workspace to partial results, on
the CPU: whatever bytes stand there (those of a run whose bounded wait gave up
before they were written), every row it reads lies in the workspace."""

import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_attention_bsa_gb300", "csrc")

SHIM = """
#include "bsa_join.h"
extern "C" void parts(int first, int last, int ctas, int segment, int two, int half, int rows, int row, int* out) {
  const bsa::Parts p = bsa::segment_parts(first, last, ctas, segment, two != 0, half, rows, row);
  out[0] = p.n; out[1] = p.at; out[2] = p.step;
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    d = tmp_path_factory.mktemp("join")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    fn = ctypes.CDLL(str(so)).parts

    def call(*args):
        out = (ctypes.c_int * 3)()
        fn(*args, out)
        return tuple(out)

    return call


STALE = [0, 1, -1, 7, 151, 152, 153, 1 << 20, (1 << 31) - 1, -(1 << 31), 0x7F7F7F7F, -0x5A5A5A5B, 0x3F800000, -0x800000]


@pytest.mark.parametrize("ctas,segments,two,half,rows", [(152, 8, 1, 0, 4), (152, 1, 1, 0, 128), (152, 4096, 0, 1, 128),
                                                         (1, 33, 0, 0, 128), (152, 64, 1, 0, 1)])
def test_any_bytes_lead_into_the_workspace_or_to_nothing(parts, ctas, segments, two, half, rows):
    r = random.Random(ctas + segments)
    pairs = [(a, b) for a in STALE for b in STALE]
    pairs += [(r.getrandbits(32) - (1 << 31), r.getrandbits(32) - (1 << 31)) for _ in range(2000)]
    pairs += [(r.randrange(ctas), r.randrange(ctas)) for _ in range(500)]
    for first, last in pairs:
        for segment in (0, segments // 2, segments - 1):
            row = r.randrange(rows)
            n, at, step = parts(first, last, ctas, segment, two, half, rows, row)
            if not 0 <= first <= last < ctas:
                assert n == 0, (first, last)
                continue
            assert n == (last - first + 1) * (2 if two else 1)
            # the workspace has two rows of each for every number segment + CTA
            assert 0 <= at and at + (n - 1) * step < (segments + ctas) * 2 * rows
            where = [at + x * step for x in range(n)]
            want = [((segment + c) * 2 + g) * rows + row for c in range(first, last + 1)
                    for g in ((0, 1) if two else (half,))]
            assert where == want
