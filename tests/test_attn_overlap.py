"""The overlap rule of the attention entry points (csrc/row_overlap.h, compiled here for the
host) against the bytes themselves."""
from __future__ import annotations

import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir,
                    "block_fp8_mixture_router_gb300", "csrc")


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("overlap")
    src, lib = d / "overlap.cc", d / "overlap.so"
    src.write_text(
        '#include "row_overlap.h"\n'
        'extern "C" int overlap(uint64_t a, int64_t as, int64_t aw, uint64_t b, int64_t bs,\n'
        '                       int64_t bw, int64_t rows) {\n'
        '  return moe::rows_overlap(a, as, aw, b, bs, bw, rows);\n'
        '}\n')
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).overlap
    f.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64] * 2 + [ctypes.c_int64]
    return f


def spans(at, stride, width, rows):
    return {at + r * stride + x for r in range(rows) for x in range(width)}


@pytest.mark.parametrize("seed", range(4))
def test_overlap_is_a_shared_byte(overlap, seed):
    r = random.Random(seed)
    seen = [0, 0]
    for _ in range(4000):
        rows = r.choice([1, 2, 3, r.randint(1, 12)])
        aw, bw = r.randint(1, 12), r.randint(1, 12)
        s = max(aw, bw) + r.choice([0, 0, 1, r.randint(0, 30)])
        a_s, b_s = (s, s) if r.random() < 0.5 else (aw + r.randint(0, 20), bw + r.randint(0, 20))
        a, b = 1000, 1000 + r.randint(-200, 200)
        want = bool(spans(a, a_s, aw, rows) & spans(b, b_s, bw, rows))
        assert bool(overlap(a, a_s, aw, b, b_s, bw, rows)) == want, (a_s, aw, b, b_s, bw, rows)
        seen[want] += 1
    assert min(seen) > 500


def test_column_ranges_of_one_buffer_share_nothing(overlap):
    for rows in (1, 2, 65536):
        for w0, w1 in ((2048, 2048), (16, 4080), (4080, 16)):
            assert not overlap(1 << 40, 4096, w0, (1 << 40) + w0, 4096, w1, rows)
            assert not overlap((1 << 40) + w0, 4096, w1, 1 << 40, 4096, w0, rows)
            assert overlap(1 << 40, 4096, w0, (1 << 40) + w0 - 1, 4096, w1, rows)
