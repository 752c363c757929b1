"""The rotation's table of turns (csrc/rope_turns.h, compiled here for the host) against the
definition in 80 decimal digits."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from turns_reference import turns

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir,
                    "block_fp8_mixture_router_gb300", "csrc")


@pytest.fixture(scope="module")
def table(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("turns")
    src, lib = d / "turns.cc", d / "turns.so"
    src.write_text(
        '#include "rope_turns.h"\n'
        'extern "C" uint64_t turns(int rot, int scaling, double base, double factor, int trained,\n'
        '                          double low, double high, int i) {\n'
        '  return moe::rope_turns(moe::RopeSpec{rot, scaling, base, factor, trained, low, high}, i);\n'
        '}\n')
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).turns
    f.restype = ctypes.c_uint64
    f.argtypes = [ctypes.c_int] * 2 + [ctypes.c_double] * 2 + [ctypes.c_int] + \
        [ctypes.c_double] * 2 + [ctypes.c_int]
    return f


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5, 1.0000001, 1e7 / 3])
@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 4.0), (1, 0.3), (2, 8.0), (2, 1.7)])
def test_turns_are_the_definition_s(table, base, rot, scaling, factor):
    """Within 0.51 units of 2^-64 of a turn: the rounding to a unit, and what is left of 106
    bits after the arithmetic."""
    for i in range(rot // 2):
        got = table(rot, scaling, base, factor, 8192, 1.0, 32.0, i)
        want = turns(rot, scaling, base, factor, 8192, 1.0, 32.0, i)  # units of 2^-64
        off = (got - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        assert off <= 0.51, (i, float(off))
