"""The one-step quotient behind bf16 rows' e4m3 codes (csrc/rows_device.cuh, div_by), in exact
arithmetic for every pair of mantissas of a value and of its group's largest, without sampling.

A quotient is 448 x / amax for mantissas x and amax in [128, 256), times a power of two that
keeps it at most 448.  In e4m3's normal range (2^-6 and more) that power changes nothing about
rounding, so one of them does for each pair; below, the steps are of one size and each power
counts, down to where every quotient is less than half of the smallest step, 2^-10."""
from __future__ import annotations

from fractions import Fraction as F

import pytest

from test_ops_division import check, e4m3, f32, scale_of

MANTISSAS = range(128, 256)


def exponents(x, amax):
    """Powers of two that a pair's quotient is checked at: one in e4m3's normal range, and
    those that lead below it and not to zeros alone."""
    first = 0 if x <= amax else 1
    return [first] + [k for k in range(1, 24) if F(1, 2048) < F(448 * x, amax * 2 ** k) < F(1, 32)]


@pytest.mark.parametrize("part", range(8))
def test_every_pair(part):
    for amax in MANTISSAS[part::8]:
        s = scale_of(F(amax))
        assert s == f32(F(amax, 448))
        for x in MANTISSAS:
            for k in exponents(x, amax):
                check(F(x, 2 ** k), s, True)


def test_the_range_covers_what_matters():
    """Every pair has one normal quotient and all that round to subnormals; what lies below the
    range is zero whatever an ulp does."""
    for x in MANTISSAS:
        for amax in MANTISSAS:
            q = F(448 * x, amax)
            ks = exponents(x, amax)
            assert F(1, 64) <= q / 2 ** ks[0] <= 448
            for k in range(1, 24):
                if F(1, 1024) <= q / 2 ** k < F(1, 64):
                    assert k in ks
            assert e4m3(q / 2 ** (ks[-1] + 1) * (1 + F(1, 2 ** 20))) == 0
