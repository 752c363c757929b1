"""Attention over pages whose value scales are far apart: a page reaches the rows that see
it by its weight times its scale, and the others not at all (needs a GB300)."""
from __future__ import annotations

import math

import pytest
import torch

import attn_reference as R
from test_gpu_attn import Case, check_close, dev, m  # noqa: F401

pytestmark = pytest.mark.gpu

LN2 = math.log(2.0)


def expected(c, q):
    """(out, tolerance) in 64 bits, all of the tolerance relative to what the row itself
    sees.  With A the weighted mean of |v| and B the largest weight x page scale of a key:
    - the output's rounding to bf16;
    - the weights' rounding to 11 bits, and the sums' in 32 bits (2 n half-steps): A times
      those; a weight below 2^-30 of the largest weight x scale lost: 448 B 2^-30 a key;
    - an error d in every score (natural units) moves a weighted mean by 2 d A: queries to
      2^-17 of their largest value, products summed in fp32 (D + 8 half-steps of sum |q k|),
      the score and the logarithm of the page's scale rounded, added and subtracted (4
      half-steps of the largest of each), the exponential and the logarithm 2^-22 each."""
    s = c.shape
    P, D, g = s.page_tokens, s.head_dim, s.q_heads // s.kv_heads
    scale = s.softmax_scale or 1.0 / math.sqrt(D)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for i, (n, kv) in enumerate(c.seqs):
        r0 = int(c.row_start[i])
        ids = c.pages[i, :-(-kv // P)].long()
        for h in range(s.kv_heads):
            ks, vs = (c.scales[x][ids, h].double().repeat_interleave(P)[:kv] for x in "kv")
            k, v = (R.decode(c.codes[x][ids, h]).reshape(-1, D)[:kv] for x in "kv")
            k, v = k * ks[:, None], v * vs[:, None]
            for t in range(n):
                pos = kv - n + t
                lo, hi = max(0, pos - s.window + 1) if s.window else 0, pos + 1
                if hi <= lo:
                    continue
                x = q[r0 + t, h * g:(h + 1) * g].double()
                sc = x @ k[lo:hi].T * scale
                w = torch.softmax(sc, -1)
                o = w @ v[lo:hi]
                A = w @ v[lo:hi].abs()
                B = (w * vs[lo:hi]).amax(-1, keepdim=True)
                size = (x.abs() @ k[lo:hi].abs().T).amax(-1) * scale
                far = sc.abs().amax(-1) + vs[lo:hi].log2().abs().max() * LN2
                d = (2.0 ** -17 * x.abs().amax(-1) * k[lo:hi].abs().sum(-1).max() * scale +
                     (D + 8) * R.HALF_FP32 * size + 4 * R.HALF_FP32 * far + 2 * 2.0 ** -22)
                out[r0 + t, h * g:(h + 1) * g] = o
                tol[r0 + t, h * g:(h + 1) * g] = (
                    R.HALF_BF16 * o.abs() + (hi - lo) * 448 * 2.0 ** -30 * B +
                    A * (R.HALF_FP16 + 2 * (hi - lo) * R.HALF_FP32 + 2 * d[:, None]))
    return out, tol


def check(c, q):
    out = c.net.forward(q, c.cache, c.batch)
    check_close(out, *expected(c, q))
    assert c.net.device_status() == m.MOE_OK
    return out


def bits(t):
    return t.contiguous().view(torch.int16)


# few rows in one tile, several tiles of the decode kernel, rows for the prompt kernel, and
# a long axis, whose keys CTAs share
FORMS = [(dict(q_heads=1, kv_heads=1, head_dim=128, page_tokens=16), 16, 40),
         (dict(q_heads=6, kv_heads=2, head_dim=64, page_tokens=16), 5, 35),
         (dict(q_heads=1, kv_heads=1, head_dim=256, page_tokens=32), 40, 90),
         (dict(q_heads=4, kv_heads=2, head_dim=128, page_tokens=32), 180, 200),
         (dict(q_heads=8, kv_heads=2, head_dim=64, page_tokens=16), 150, 150),
         (dict(q_heads=8, kv_heads=4, head_dim=256, page_tokens=64), 140, 300),
         (dict(q_heads=4, kv_heads=1, head_dim=128, page_tokens=64), 4, 4994),
         (dict(q_heads=8, kv_heads=1, head_dim=128, page_tokens=64), 150, 5000)]


@pytest.mark.parametrize("kw,rows,tokens", FORMS)
@pytest.mark.parametrize("window", [0, 12])
@pytest.mark.parametrize("up", [40, 100])
def test_rows_that_do_not_see_a_page_do_not_feel_it(dev, kw, rows, tokens, window, up):  # noqa: F811
    """The page that some rows of the batch see and others do not (yet, or no longer): with
    value and key scales 2^up larger, and with any codes, the others' bits are the same."""
    shape = m.AttnShape(rotary_dim=0, window=window, **kw)
    P = shape.page_tokens
    c = Case(dev, shape, [(rows, tokens)], seed=rows + window)
    q = c.q()
    plain = check(c, q).clone()
    j = (tokens - (rows + 1) // 2) // P                        # from the middle row on
    page = int(c.pages[0, j])
    pos = torch.arange(tokens - rows, tokens, device=dev)
    low = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
    blind = (pos < j * P) | (low >= (j + 1) * P)
    assert bool(blind.any()) and not bool(blind.all())
    c.scales["v"][page] = 2.0 ** (up - 7)
    big = check(c, q).clone()
    assert torch.equal(bits(big[blind]), bits(plain[blind]))
    c.scales["k"][page] = 2.0 ** (up - 7)
    c.codes["k"][page] = 0x7E
    c.codes["v"][page] = 0x7F
    out = c.net.forward(q, c.cache, c.batch)
    assert torch.equal(bits(out[blind]), bits(plain[blind]))
    assert bool(torch.isnan(out[~blind]).all())


@pytest.mark.parametrize("kw,rows,tokens", FORMS)
@pytest.mark.parametrize("up,below", [(35, 60), (150, 40), (200, 190), (90, 5)])
def test_large_pages_of_low_weight(dev, kw, rows, tokens, up, below):  # noqa: F811
    """All rows see a page whose value scale is 2^up of the others' and whose weights are
    about 2^-below of theirs: what counts of it depends on both."""
    shape = m.AttnShape(rotary_dim=0, softmax_scale=0.5, **kw)
    c = Case(dev, shape, [(rows, tokens)], seed=up)
    q = c.q()
    q[..., 0] = 64.0
    P = shape.page_tokens
    first = max(tokens - rows, 1)
    low = min(3, (first - 1) // P) if first > P else 0         # seen by (nearly) all rows
    page = int(c.pages[0, low])
    e = -100 if up > 90 else -8
    c.scales["v"].fill_(2.0 ** e)
    c.scales["v"][page] = 2.0 ** (e + up)
    c.scales["k"].fill_(2.0 ** -9)                             # scores of a few units
    c.codes["k"][..., 0] = 0
    # 64 x code x 2^-9 x 0.5 natural units
    code = R.encode(torch.tensor([-min(below * LN2 * 16, 448.0)], dtype=torch.float64)).to(dev)
    if below * LN2 * 16 > 448.0:                               # (further down by a larger scale)
        c.scales["k"][page] = 2.0 ** -9 * below * LN2 * 16 / 448.0
    c.codes["k"][page, :, :, 0] = code
    check(c, q)


@pytest.mark.parametrize("kw,rows,tokens", FORMS)
def test_scales_of_the_whole_range(dev, kw, rows, tokens):  # noqa: F811
    """Value scales anywhere from 2^-100 to 2^100, page by page."""
    shape = m.AttnShape(rotary_dim=0, **kw)
    c = Case(dev, shape, [(rows, tokens)], seed=9)
    n = c.scales["v"].shape
    for _ in range(3):
        e = torch.randint(-100, 101, n, generator=c.g, device=dev)
        c.scales["v"].copy_(torch.exp2(e.float()))
        check(c, c.q())
    for e in (-100, 100):
        c.scales["v"].fill_(2.0 ** e)
        check(c, c.q())


@pytest.mark.parametrize("rows,tokens", [(1, 100), (3, 700), (150, 400), (1, 6000), (150, 5000)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 20, 2.0 ** 100, 2.0 ** 124])
def test_zero_tokens_keep_their_weight(dev, rows, tokens, size):  # noqa: F811
    """Pages of zeros, which the append gives the smallest scale there is, beside pages of
    ordinary and of large values: their keys count in the softmax all the same."""
    shape = m.AttnShape(q_heads=4, kv_heads=2, head_dim=128, page_tokens=16, rotary_dim=0)
    c = Case(dev, shape, [(rows, tokens)], seed=17, max_rows=tokens)
    k, v = c.randn(tokens, 2, 128), c.randn(tokens, 2, 128) * size
    at = torch.arange(tokens, device=dev) // 16
    v[(at % 3 != 0)] = 0
    fill = m.AttnBatch(torch.tensor([0, tokens], dtype=torch.int32, device=dev), c.kv_len, c.pages,
                       tokens)
    c.net.append(k, v, c.cache, fill)
    assert float(c.scales["v"].nan_to_num(1.0).min()) == 2.0 ** -100
    check(c, c.q())
