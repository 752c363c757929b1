"""The quotients behind the rows' e4m3 codes (csrc/rows_device.cuh, div_by), restated in exact
rational arithmetic: two steps give the IEEE quotient, one step gives its e4m3 code for every
pair of bf16 value and bf16 largest value."""
from __future__ import annotations

import random
from fractions import Fraction as F


def rounded(x: F, bits: int) -> F:
    """To `bits` significant bits, ties to even (no exponent limits)."""
    if x == 0:
        return x
    a = abs(x)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    if F(2) ** e > a:
        e -= 1
    u = F(2) ** (e - bits + 1)
    n, r = divmod(a / u, 1)
    if r > F(1, 2) or (r == F(1, 2) and n % 2):
        n += 1
    return n * u if x > 0 else -n * u


def f32(x: F) -> F:
    return rounded(x, 24)


def e4m3(x: F) -> F:
    if abs(x) >= F(1, 64):
        y = rounded(x, 4)
        return min(max(y, F(-448)), F(448))
    n, r = divmod(abs(x) * 512, 1)       # subnormals: multiples of 2^-9
    if r > F(1, 2) or (r == F(1, 2) and n % 2):
        n += 1
    return F(n, 512) if x > 0 else -F(n, 512)


def fma(a, b, c):
    return f32(a * b + c)


def step(q, v, s, y):
    return fma(fma(-q, s, v), y, q)


RECIP448 = f32(F(1, 448))


def scale_of(amax: F) -> F:
    q = f32(amax * RECIP448)
    return step(step(q, amax, F(448), RECIP448), amax, F(448), RECIP448)


def check(v, s, short: bool):
    y = f32(1 / s)
    one = step(f32(v * y), v, s, y)
    want = f32(v / s)
    assert step(one, v, s, y) == want
    if short:
        assert e4m3(one) == e4m3(want), (v, s)


def test_every_pair_of_bf16_mantissas():
    for amax in range(128, 256):
        s = scale_of(F(amax))
        assert s == f32(F(amax, 448))
        for x in range(128, 256):
            if x <= amax:
                check(F(x), s, True)
        for x in range(128 + amax % 7, 256, 7):      # e4m3's subnormals, and below
            for k in (1, 13, 14, 15, 16, 17):
                check(-F(x, 2 ** k), s, True)


def test_fp32_values():
    rng = random.Random(0)
    for _ in range(3000):
        amax = F(rng.randrange(1 << 23, 1 << 24))
        s = scale_of(amax)
        assert s == f32(amax / 448)
        check(F(rng.randrange(1 << 23, int(amax) + 1), 2 ** rng.randrange(0, 12)), s, False)
        # beside the midpoints of e4m3, where a wrong last bit changes the code
        c = F(2 * rng.randrange(8, 16) + 1, 2)
        v = f32(s * c)
        for d in (-1, 0, 1):
            check(v * (1 + d * F(1, 2 ** 23)) if d else v, s, False)


def test_the_check_sees_a_missing_step():
    """A quotient without its last step is not the IEEE one."""
    wrong = 0
    for amax in range(129, 256, 2):
        s = scale_of(F(amax))
        y = f32(1 / s)
        wrong += any(f32(F(x) * y) != f32(F(x) / s) for x in range(128, amax))
    assert wrong > 32
