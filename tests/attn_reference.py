"""Plain 64-bit forms of the attention operators, and how far a kernel may be off.

The forms follow the definitions in include/moe.h sequence by sequence; nothing
here shares code with the library.  A tolerance counts the roundings that the
operator's definition and its kernels make; each is derived beside its form.
"""
from __future__ import annotations

import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_FP16 = torch.finfo(torch.float16).eps / 2
HALF_FP32 = torch.finfo(torch.float32).eps / 2
MIN_EXP = -100
NAN_CODE = 0x7F


def e4m3_table():
    """Value of every e4m3 code, 64 bits."""
    c = torch.arange(256)
    s, e, m = c // 128, (c // 8) % 16, (c % 8).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    v = torch.where(s == 1, -v, v)
    v[NAN_CODE] = v[NAN_CODE | 128] = float("nan")
    return v


def decode(codes):
    return e4m3_table().to(codes.device)[codes.long()]


def encode(x):
    """Nearest e4m3 code of 64-bit values with |x| <= 448, ties to the even code."""
    t = e4m3_table()[:NAN_CODE].to(x.device)
    mid = (t[1:] + t[:-1]) / 2
    a = x.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    code = torch.where(lo == hi, lo, lo + lo % 2)
    neg = torch.signbit(x).long() * 128
    return (code + neg).to(torch.uint8)


def block_scale(amax: float) -> float:
    """The smallest 2^k with 448 * 2^k >= amax, k >= MIN_EXP."""
    k = MIN_EXP
    while math.ldexp(448.0, k) < amax:
        k += 1
    return math.ldexp(1.0, k)


def frequencies(shape):
    rot = shape.rotary_dim
    f = shape.rope_base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))
    if shape.rope_scaling == "linear":
        f = f / shape.rope_factor
    if shape.rope_scaling == "by_parts":
        t = shape.rope_trained_positions * f / (2 * math.pi)
        g = ((t - shape.rope_turns_low) / (shape.rope_turns_high - shape.rope_turns_low))
        g = g.clamp(0.0, 1.0)
        f = f * (g + (1 - g) / shape.rope_factor)
    return f


def rope(shape, x, positions, gamma=None, eps=1e-6):
    """(y, tolerance) of moe_rope on x [rows, heads, D]; CPU, 64 bits.

    Tolerance: the rounding to bf16; the norm's fp32 sum and products (relative
    D + 8 half-steps of fp32, far below 2^-14 of the value for D <= 256); the
    angle (2^-25 of a turn, 2 pi times that in radians) and the two functions
    (2^-21 each at most), relative to the pair's magnitudes."""
    x = x.double().cpu()
    D = x.shape[-1]
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double().cpu()
    rot = shape.rotary_dim
    half = rot // 2
    i = torch.arange(half)
    one = i if shape.rope_layout == "half" else 2 * i
    two = i + half if shape.rope_layout == "half" else 2 * i + 1
    angle = positions.double().cpu()[:, None] * frequencies(shape)[None]
    angle = torch.remainder(angle, 2 * math.pi)[:, None, :]
    c, s = torch.cos(angle) * shape.rope_amplitude, torch.sin(angle) * shape.rope_amplitude
    y = x.clone()
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    size = x.abs()
    pair = (a.abs() + b.abs()) * shape.rope_amplitude
    size[..., one], size[..., two] = pair, pair
    # positions in fp32-free 64-bit arithmetic: |position| x 2^-53 radians, below 2^-20 here
    tol = HALF_BF16 * y.abs() + size * ((D + 8) * HALF_FP32 * (gamma is not None) +
                                        2 * math.pi * 2.0 ** -25 + 2.0 ** -21 + 2.0 ** -20)
    return y, tol


def append(shape, codes, scales, pages, row_start, kv_len, x):
    """moe_kv_append of x [rows, kv_heads, D] into (codes, scales), CPU tensors that are
    changed in place; exact: every step is one rounding of an exact quotient."""
    P = shape.page_tokens
    for s in range(len(kv_len)):
        r0, r1 = int(row_start[s]), int(row_start[s + 1])
        first = int(kv_len[s]) - (r1 - r0)
        start = max(first, 0)
        for j in range(start // P, -(-int(kv_len[s]) // P)):
            lo, hi = max(start, j * P), min(int(kv_len[s]), (j + 1) * P)
            if lo >= hi:
                continue
            page = int(pages[s, j])
            rows = x[r0 + lo - first:r0 + hi - first]
            for h in range(x.shape[1]):
                v = rows[:, h].double()
                fine = torch.isfinite(v).all(-1)
                amax = float(v[fine].abs().max()) if bool(fine.any()) else 0.0
                scale = block_scale(amax)
                slot = lo - j * P
                if slot:
                    old = float(scales[page, h])
                    scale = max(scale, old)
                    if scale > old:
                        kept = decode(codes[page, h, :slot]) * (old / scale)
                        again = encode(torch.nan_to_num(kept))
                        codes[page, h, :slot] = torch.where(torch.isnan(kept),
                                                            torch.full_like(again, NAN_CODE), again)
                new = encode(torch.where(fine[:, None], v, torch.zeros_like(v)) / scale)
                new[~fine] = NAN_CODE
                codes[page, h, slot:slot + hi - lo] = new
                scales[page, h] = scale


def attention(shape, q, codes_k, scales_k, codes_v, scales_v, pages, row_start, kv_len):
    """(out, tolerance) of moe_attn_forward; 64 bits, on q's device.

    Tolerance, with A the weighted mean of |v|, per row:
    - the output's rounding to bf16;
    - the weights' rounding to 11 bits (relative HALF_FP16 each, so A times that), and
      the smallest of them lost: 2^-30 of the largest value for each key;
    - the scores: the queries are off by up to 2^-17 of their largest value, the products
      accumulate in fp32 (D + 8 half-steps of sum |q k|), the score in log2 units is
      rounded and subtracted in fp32 (4 half-steps of the largest), and the exponential
      is good to 2^-22; an error d in every score moves a weighted mean by at most
      2 d A (natural units)."""
    P, D, g = shape.page_tokens, shape.head_dim, shape.q_heads // shape.kv_heads
    scale = shape.softmax_scale or 1.0 / math.sqrt(D)
    dev = q.device
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    for s in range(len(kv_len)):
        r0, r1, n_keys = int(row_start[s]), int(row_start[s + 1]), int(kv_len[s])
        n = r1 - r0
        if n == 0 or n_keys == 0:
            continue
        ids = pages[s, :-(-n_keys // P)].long()
        pos = torch.arange(n_keys - n, n_keys, device=dev)
        j = torch.arange(n_keys, device=dev)
        see = j[None] <= pos[:, None]
        if shape.window:
            see &= j[None] > pos[:, None] - shape.window
        for h in range(shape.kv_heads):
            k = (decode(codes_k[ids, h]) * scales_k[ids, h].double()[:, None, None])
            v = (decode(codes_v[ids, h]) * scales_v[ids, h].double()[:, None, None])
            k, v = k.reshape(-1, D)[:n_keys], v.reshape(-1, D)[:n_keys]
            # tokens that a row does not see reach it in no way, whatever they hold
            for i in range(n):
                m = see[i]
                if not bool(m.any()):
                    continue
                x = q[r0 + i, h * g:(h + 1) * g].double()              # [g, D]
                sc = x @ k[m].T * scale
                w = torch.softmax(sc, -1)
                o = w @ v[m]
                out[r0 + i, h * g:(h + 1) * g] = o
                A = w @ v[m].abs()
                size = (x.abs() @ k[m].abs().T).amax(-1) * scale
                d = (2.0 ** -17 * x.abs().amax(-1) * k[m].abs().sum(-1).max() * scale +
                     (D + 8) * HALF_FP32 * size +
                     4 * HALF_FP32 * sc.abs().amax(-1) * 1.4427 + 2.0 ** -22)
                tol[r0 + i, h * g:(h + 1) * g] = (
                    HALF_BF16 * o.abs() + A * (HALF_FP16 + 2 * d[:, None]) +
                    int(m.sum()) * 2.0 ** -30 * v[m].abs().max())
    return out, tol
