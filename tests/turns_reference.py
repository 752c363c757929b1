"""Turns per position of a rotation's pairs from their definition, in 80 decimal digits."""
from __future__ import annotations

from decimal import Decimal, getcontext

getcontext().prec = 80

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turns(rot, scaling, base, factor, trained, low, high, i) -> Decimal:
    """base^(-2i/rot) / 2 pi with the scaling (0 plain, 1 linear, 2 by parts), in units of
    2^-64 of a turn."""
    t = (-Decimal(2 * i) / Decimal(rot) * Decimal(base).ln()).exp() / (2 * PI)
    if scaling == 1:
        t /= Decimal(factor)
    if scaling == 2:
        g = (t * trained - Decimal(low)) / (Decimal(high) - Decimal(low))
        g = min(Decimal(1), max(Decimal(0), g))
        t *= g + (1 - g) / Decimal(factor)
    return t * 2 ** 64
