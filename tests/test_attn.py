"""The attention entry points without a GPU: refusals, and the arithmetic by which
the kernels number their work, restated (coverage, no slot used twice, bounds)."""
from __future__ import annotations

import ctypes
import math
import random

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe
from attn_reference import block_scale, decode, encode, frequencies
from block_fp8_mixture_router_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return moe.load_library()


def config(**kw):
    s = moe.AttnShape(**{k: v for k, v in kw.items() if k not in ("max_rows", "max_seqs", "cap")})
    return s.config(kw.get("max_rows", 64), kw.get("max_seqs", 4), kw.get("cap", 0))


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(head_dim=0), dict(kv_heads=0), dict(kv_heads=65, q_heads=65),
    dict(q_heads=15), dict(q_heads=34), dict(q_heads=1, kv_heads=2), dict(page_tokens=8),
    dict(page_tokens=48), dict(page_tokens=256), dict(rotary_dim=3), dict(rotary_dim=130),
    dict(rotary_dim=-2), dict(rope_base=1.0), dict(rope_base=float("nan")),
    dict(rope_amplitude=0.0), dict(rope_scaling="linear", rope_factor=0.0),
    dict(rope_scaling="by_parts", rope_factor=4.0),
    dict(rope_scaling="by_parts", rope_factor=4.0, rope_trained_positions=8,
         rope_turns_low=2.0, rope_turns_high=2.0),
    dict(softmax_scale=-1.0), dict(softmax_scale=float("inf")), dict(window=-1),
    dict(max_rows=0), dict(max_rows=65537), dict(max_seqs=0), dict(max_seqs=4097)])
def test_unsupported_shapes_are_refused(bad):
    cfg = config(**bad)
    rc, h = moe.moe_attn_create(cfg, 0)
    assert rc == moe.MOE_ERR_UNSUPPORTED_SHAPE and not h.value
    assert moe.moe_attn_required_bytes(cfg)[0] == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_bytes_cap_and_null_arguments():
    rc, n = moe.moe_attn_required_bytes(config())
    assert rc == moe.MOE_OK and n > 64 * 16 * 128 * 2
    rc, h = moe.moe_attn_create(config(cap=1 << 16), 0)
    assert rc == moe.MOE_ERR_ALLOC_LIMIT and not h.value
    assert moe.moe_attn_create(config(), -1)[0] == moe.MOE_ERR_INVALID_ARG
    bad = moe.MOE_ERR_INVALID_ARG
    assert moe.moe_rope(None, None, 0, 1, None, None, 1e-6, 1, None, 0, 0) == bad
    assert moe.moe_kv_append(None, None, None, 0, None, 0, None, 0) == bad
    assert moe.moe_attn_forward(None, None, None, 0, None, None, 0, 0) == bad
    assert moe.moe_attn_step(None, None, None, 0, None, None, 1e-6, None, None, 0, 0) == bad
    assert moe.moe_attn_last_device_status(None) == bad
    moe.moe_attn_destroy(None)
    with pytest.raises(ValueError):
        moe.AttnShape(rope_layout="third").config(1, 1)


def test_struct_layouts_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    kinds = {"moe_attn_config": moe.moe_attn_config, "moe_kv_cache": moe.moe_kv_cache,
             "moe_attn_batch": moe.moe_attn_batch}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "moe.h"', "int main(void) {"]
    for st, cls in kinds.items():
        lines.append(f'  printf("{st} size %zu\\n", sizeof({st}));')
        lines += [f'  printf("{st} {n} %zu\\n", offsetof({st}, {n}));' for n, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {tuple(ln.split()[:2]): int(ln.split()[2]) for ln in out if ln.strip()}
    for st, cls in kinds.items():
        assert got[(st, "size")] == ctypes.sizeof(cls)
        for n, _ in cls._fields_:
            assert got[(st, n)] == getattr(cls, n).offset, (st, n)


def test_fixed_point_turns_are_exact_at_far_positions():
    """position x round(f / 2 pi x 2^64) modulo 2^64 as a signed fraction of a turn is
    within |position| x 2^-65 + 2^-53 relative error of the frequency itself."""
    f = frequencies(moe.AttnShape(rotary_dim=128))
    for i in (0, 1, 17, 63):
        turns = float(f[i]) / (2 * math.pi)
        frac = int(math.floor(turns % 1.0 * 2.0 ** 32))
        low = round((turns % 1.0 * 2.0 ** 32 - frac) * 2.0 ** 32)
        entry = (frac << 32) + low
        for pos in (0, 1, -1, 4095, 10 ** 6 + 7, -(10 ** 6), 2 ** 31 - 1, -(2 ** 31)):
            t = (pos * entry) % 2 ** 64
            signed = t - 2 ** 64 if t >= 2 ** 63 else t
            from fractions import Fraction
            exact = Fraction(turns) * pos
            off = Fraction(signed, 2 ** 64) - exact
            off -= round(off)
            assert abs(off) <= Fraction(abs(pos), 2 ** 65), (i, pos)


def test_block_scale_from_the_bits():
    """The kernel takes the exponent from amax's bits: mantissa above 1.75 (448 = 1.75 x
    2^8) takes the next power of two."""
    import struct
    r = random.Random(5)
    values = [448.0, 448.1, 447.9, 1.0, 0.875, 1.75, 1.7500001, 3e38, 1e-30, 1e-38]
    values += [math.ldexp(r.uniform(1, 2), r.randint(-90, 120)) for _ in range(200)]
    for a in values:
        u = struct.unpack("<I", struct.pack("<f", a))[0]
        a = struct.unpack("<f", struct.pack("<I", u))[0]
        k = max((u >> 23) - 127 - 8 + ((u & 0x7FFFFF) > 0x600000), -100)
        assert math.ldexp(1.0, k) == block_scale(a), a
    assert block_scale(0.0) == 2.0 ** -100


def test_reference_codes_are_torch_s_rounding():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.05, 0.05, 4001)])
    mine = encode(x.double())
    torch_s = x.to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(decode(mine), decode(torch_s))


def unit_seq(row_start, n_seqs, rows, per, extra, u):
    below = sum(1 for s in range(1, n_seqs)
                if min(max(row_start[s], 0), rows) // per + extra * s <= u)
    return below, min(max(row_start[below], 0), rows) // per + extra * below


@pytest.mark.parametrize("seed", range(6))
def test_every_page_and_row_tile_has_one_unit(seed):
    """Sequence s's units begin at row_start[s] / per + extra s: with extra 2 every page
    that a sequence's rows reach, with extra 1 every row tile, gets exactly one unit."""
    r = random.Random(seed)
    n = r.choice([1, 2, 7, 40])
    lens = [r.choice([0, 1, 1, r.randint(0, 300)]) for _ in range(n)]
    ctx = [r.choice([0, r.randint(0, 500)]) for _ in range(n)]
    start = [0]
    for k in lens:
        start.append(start[-1] + k)
    rows = start[-1]
    for P in (16, 64, 128):
        seen = {}
        for u in range(rows // P + 2 * n):
            s, u0 = unit_seq(start, n, rows, P, 2, u)
            if lens[s] == 0 or u < u0:
                continue
            j = ctx[s] // P + (u - u0)
            if max(ctx[s], j * P) < min(ctx[s] + lens[s], (j + 1) * P):
                assert (s, j) not in seen
                seen[(s, j)] = u
        assert set(seen) == {(s, j) for s in range(n) if lens[s]
                             for j in range(ctx[s] // P, (ctx[s] + lens[s] - 1) // P + 1)}
    for tq in (1, 3, 8, 16, 42, 128):
        seen = set()
        for u in range(rows // tq + n):
            s, u0 = unit_seq(start, n, rows, tq, 1, u)
            t = u - u0
            if t >= 0 and t * tq < lens[s]:
                assert (s, t) not in seen
                seen.add((s, t))
        assert seen == {(s, t) for s in range(n) for t in range(-(-lens[s] // tq))}


@pytest.mark.parametrize("seed", range(8))
def test_equal_runs_cover_every_tile_and_no_slot_twice(seed):
    """The decode grid deals the key tiles of all units to the CTAs in equal runs: every
    tile is worked once, a unit's parts are as many as counted, and no two parts of a launch
    lie in one slot."""
    r = random.Random(100 + seed)
    widths = [r.choice([1, 2, r.randint(1, 400)]) for _ in range(r.randint(1, 60))]
    total, grid = sum(widths), r.choice([1, 2, 7, 64, 456])
    per = -(-total // grid)
    firsts = [sum(widths[:i]) for i in range(len(widths))]
    worked, slots, parts, counters = [0] * total, set(), {}, {}
    for cta in range(grid):
        at, end = per * cta, min(per * cta + per, total)
        while at < end:
            i = max(k for k in range(len(firsts)) if firsts[k] <= at)
            stop = min(end, firsts[i] + widths[i])
            for t in range(at, stop):
                worked[t] += 1
            c0, c1 = firsts[i] // per, (firsts[i] + widths[i] - 1) // per
            if not (at == firsts[i] and stop == firsts[i] + widths[i]):
                slot = 2 * c0 + 1 if at == firsts[i] else 2 * cta
                assert slot not in slots and slot < 2 * grid
                slots.add(slot)
                # where the merge will look for it
                assert slot == (2 * c0 + 1 if cta == c0 else 2 * (c0 + (cta - c0)))
                parts.setdefault(i, []).append(cta)
                assert counters.setdefault(c0, i) == i
            at = stop
    assert worked == [1] * total
    for i, ctas in parts.items():
        assert ctas == list(range(firsts[i] // per, (firsts[i] + widths[i] - 1) // per + 1))
