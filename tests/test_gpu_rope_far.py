"""Rotary positions as far out as a position goes (needs a GB300)."""
from __future__ import annotations

import math

import pytest
import torch

import attn_reference as R
from test_gpu_attn import dev, m  # noqa: F401
from turns_reference import turns

pytestmark = pytest.mark.gpu

SCALINGS = {"plain": 0, "linear": 1, "by_parts": 2}


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("sign", [1, -1])
def test_angles_of_far_positions(dev, scaling, sign):  # noqa: F811
    """Pairs (1, 0) at positions near 2^31 where a pair has turned by nearly a whole number
    of half turns: the sine is the angle itself, and its relative error shows the angle's
    absolute one.  Tolerance: the angle, 1.25 x 2^-32 of a turn; the sine's fp32 arithmetic
    near zero, relative 2^-22; the rounding to bf16."""
    rot, base, factor = 128, 10000.0, 8.0
    shape = m.AttnShape(q_heads=1, kv_heads=1, head_dim=128, rotary_dim=rot, rope_base=base,
                        rope_scaling=scaling, rope_factor=factor, rope_trained_positions=8192,
                        rope_turns_low=1.0, rope_turns_high=32.0)
    net = m.Attention(shape, max_rows=1)
    entries = [turns(rot, SCALINGS[scaling], base, factor, 8192, 1.0, 32.0, i)
               for i in range(rot // 2)]
    far = [2 ** 31 - 1 - k for k in range(1 << 14)]
    picked = []  # (position, pair)
    for i in range(0, rot // 2, 3):
        e = int(entries[i].to_integral_value())

        def off(p, e=e):
            h = p * e % 2 ** 63
            return min(h, 2 ** 63 - h)
        picked += [(sign * p, i) for p in sorted(far, key=off)[:6]]
    pos = torch.tensor([p for p, _ in picked], dtype=torch.int64).to(torch.int32)
    x = torch.zeros((len(picked), 1, 128), dtype=torch.bfloat16)
    x[:, 0, :rot // 2] = 1
    y = net.rope(x.to(dev), pos.to(dev)).cpu().double()
    for row, (p, i) in enumerate(picked):
        t = (entries[i] * p) % 2 ** 64
        t = float(t if t < 2 ** 63 else t - 2 ** 64) / 2.0 ** 64
        want = math.sin(2 * math.pi * t)
        tol = (2 * math.pi * 1.25 * 2.0 ** -32 + abs(want) * (2.0 ** -22 + R.HALF_BF16) * 1.001)
        assert abs(float(y[row, 0, i + rot // 2]) - want) <= tol, (p, i, want)
