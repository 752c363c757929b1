"""The attention kernels' index arithmetic and operand splits, restated without a GPU:
swizzles, masks of a tile, shares of the keys, the layout in which parts are joined, and
how exactly queries and weights are held in 8-bit parts."""
from __future__ import annotations

import math
import random

import pytest
import torch


def swz(wide: bool, row: int, b: int) -> int:
    col = b >> 4
    if wide:
        return row * 128 + ((col ^ (row & 7)) << 4) + (b & 15)
    return row * 64 + ((col ^ ((row >> 1) & 3)) << 4) + (b & 15)


@pytest.mark.parametrize("wide", [True, False])
def test_swizzles_use_each_byte_once_and_spread_the_rows(wide):
    width = 128 if wide else 64
    at = [swz(wide, r, b) for r in range(128) for b in range(width)]
    assert sorted(at) == list(range(128 * width))
    # the same 16 bytes of eight rows one after the other lie in eight different quarters of
    # the 128 bytes that shared memory serves at once
    for b in range(0, width, 16):
        for r0 in range(0, 128, 8):
            assert len({swz(wide, r0 + i, b) % 128 // 16 for i in range(8)}) == 8


def test_rows_divide_by_the_group_without_a_division():
    for g in range(1, 17):
        for r in range(128):
            assert r * (65536 // g + 1) >> 16 == r // g


def row_mask(low, high, absent, poison):
    full = (1 << 64) - 1
    seen = 0 if high < 0 else full if high >= 63 else (2 << high) - 1
    seen &= full if low <= 0 else 0 if low > 63 else (full << low) & full
    for g in range(4):
        if (absent >> g) & 1:
            seen &= ~(0xFFFF << 16 * g)
    return seen, seen & poison


def test_row_mask_is_the_columns_seen():
    r = random.Random(3)
    for _ in range(4000):
        low, high = r.randint(-200, 200), r.randint(-200, 200)
        absent, poison = r.randint(0, 255), r.getrandbits(64)
        seen, nan = row_mask(low, high, absent, poison)
        for c in range(64):
            want = low <= c <= high and not (absent >> (c // 16)) & 1
            assert (seen >> c) & 1 == want
            assert (nan >> c) & 1 == (want and (poison >> c) & 1)


@pytest.mark.parametrize("seed", range(6))
def test_shares_of_the_keys_cover_each_tile_once(seed):
    r = random.Random(seed)
    for _ in range(300):
        lo = r.choice([0, r.randint(0, 5000)])
        hi = lo + r.choice([0, 1, r.randint(0, 3000)])
        splits = r.randint(1, 160)
        k0 = lo // 128
        n = max(-(-hi // 128), k0 + 1) - k0
        tiles = []
        for part in range(splits):
            t0, t1 = k0 + n * part // splits, k0 + n * (part + 1) // splits
            tiles += range(t0, t1)
        assert tiles == list(range(k0, k0 + n))  # some shares may be empty
        assert all(k0 * 128 <= k < (k0 + n) * 128 for k in (lo, max(hi - 1, lo)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("few", [True, False])
def test_joining_threads_read_what_was_left(D, few):
    """Every (row, column) of a part is written once, by the row's thread, and read once per
    part, by one thread of the join; threads of a row side by side read side by side."""
    tiles = 1 if D == 256 else 2
    rows, runs = (8, 1) if few else (4, 4)
    threads = D // 4 * rows * runs
    assert threads <= 1024 and 128 % rows == 0
    written = {}
    for tile in range(tiles):
        for row in range(128):
            for c in range(0, D, 4):
                at = tile * 128 * D + c * 128 + 4 * row
                assert at % 4 == 0 and at // 4 not in written
                written[at // 4] = (tile * 128 + row, c)
    assert sorted(written) == list(range(tiles * 128 * D // 4))
    read = set()
    for block in range(tiles * 128 // rows):
        row0 = block * rows
        tile = row0 >> 7
        for tid in range(D // 4 * rows):  # run 0
            row, col = row0 + tid % rows, tid // rows
            at = tile * 128 * (D // 4) + col * 128 + (row & 127)
            assert written[at] == (row, 4 * col) and at not in read
            read.add(at)
    assert len(read) == len(written)
    # a run's parts, eight (two) at a time, are each taken once
    for parts in (1, 2, 15, 16, 17, 31, 33, 148, 160):
        ahead = 2 if few else 8
        if few and parts > 16:
            continue
        taken = [p0 + k * runs for run in range(runs) for p0 in range(run, parts, ahead * runs)
                 for k in range(ahead) if p0 + k * runs < parts]
        assert sorted(taken) == list(range(parts))


def test_queries_split_into_two_e4m3_values():
    """Values scaled so that a row's largest lies in [128, 256): exact down to 1/4, and to
    2^-10, half of e4m3's smallest step, below."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).double()
    x = x[torch.isfinite(x) & (x.abs() < 256)]
    e4m3 = torch.float8_e4m3fn
    hi = x.float().to(e4m3).float()
    lo = (x.float() - hi).to(e4m3).float()
    off = (x - hi.double() - lo.double()).abs()
    assert bool((off[x.abs() >= 0.25] == 0).all())
    assert bool((off <= 2.0 ** -10).all())


def test_weights_split_into_four_e5m2_values():
    """Three bits from the top, four times, the last rounded: 11 bits of a weight, and 2^-30
    of a weight of one (2^12) where parts end as e5m2 subnormals."""
    g = torch.Generator().manual_seed(1)
    p = torch.exp2(torch.rand(200000, generator=g, dtype=torch.float64) * 60 - 45).float()
    p = torch.cat([p, torch.exp2(torch.arange(-40, 16).float()), torch.zeros(1)])
    p = p[p <= 2.0 ** 15]
    rest, total = p.clone(), torch.zeros(p.numel(), dtype=torch.float64)
    for i in range(4):
        part = rest.clone()
        if i < 3:
            part = (rest.view(torch.int32) & -0x200000).view(torch.float32)
        if i == 0:
            part = torch.where(rest < 2.0 ** -14, torch.zeros_like(part), part)
        rest = (rest - part) * 8.0
        total += part.to(torch.float8_e5m2).double() * 2.0 ** (-3 * i)
    off = (p.double() - total).abs()
    assert bool((off <= p.double() * 2.0 ** -11 + 2.0 ** (12 - 30)).all())


def test_sine_and_cosine_of_a_turn_in_32_bits():
    """A quarter turn taken out in integers, Taylor's series in fp32 for the rest, whose
    angle is held in two parts: within 2^-23 of the functions everywhere (2^-25 each for
    the last sum, the square, the series' sum and its next term)."""
    g = torch.Generator().manual_seed(2)
    t = torch.randint(0, 1 << 32, (400000,), generator=g)
    edges = torch.arange(8)[:, None] * (1 << 29) + torch.arange(-3, 4)
    t = torch.cat([t, edges.flatten() % (1 << 32)])
    u = (t + 0x20000000) & 0xFFFFFFFF
    quarter = u >> 30
    left = (u & 0x3FFFFFFF) - 0x20000000
    f32 = torch.float32

    def fma(a, b, c):
        c = c if torch.is_tensor(c) else torch.tensor(c, dtype=f32)
        return (a.double() * b.double() + c.double()).to(f32)
    unit = torch.tensor(float.fromhex("0x1.921fb6p-30"), dtype=f32)
    low = torch.tensor(float.fromhex("-0x1.777a5cp-55"), dtype=f32)
    assert abs(unit.double() + low.double() - 2 * math.pi / 2 ** 32) <= 2.0 ** -75
    n = left.to(f32)
    x = n * unit
    y = fma(n, unit, -x) + fma(n, low, (left - n.long()).to(f32) * unit)
    x2 = x * x
    one = torch.ones_like(x)
    p = fma(x2, fma(x2, fma(x2, one / 362880, -1 / 5040), 1 / 120), -1 / 6)
    s0 = x + fma(x * x2, p, y)
    q = fma(x2, fma(x2, fma(x2, fma(x2, -one / 3628800, 1 / 40320), -1 / 720), 1 / 24), -0.5)
    c0 = one + fma(x2, q, -x * y)
    odd = (quarter & 1) == 1
    c, s = torch.where(odd, s0, c0), torch.where(odd, c0, s0)
    c = torch.where(((quarter + 1) & 2) != 0, -c, c).double()
    s = torch.where((quarter & 2) != 0, -s, s).double()
    a = t.double() * (2 * math.pi / 2 ** 32)
    assert float((c - torch.cos(a)).abs().max()) <= 2.0 ** -23
    assert float((s - torch.sin(a)).abs().max()) <= 2.0 ** -23
