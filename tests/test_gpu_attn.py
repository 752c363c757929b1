"""The attention operators on the GPU against their plain 64-bit forms
(tests/attn_reference.py), at the sizes and masks where they can go wrong (needs a
GB300)."""
from __future__ import annotations

import pytest
import torch

import attn_reference as R

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


class Case:
    """Sequences of (rows, tokens) with a paged cache whose unused memory is NaN."""

    def __init__(self, dev, shape, seqs, seed=0, spare=2, hints=True, max_rows=None):
        self.shape, self.seqs, self.dev = shape, seqs, dev
        g = self.g = gen(dev, seed)
        P, D, H = shape.page_tokens, shape.head_dim, shape.kv_heads
        need = [-(-k // P) for _, k in seqs]
        n_pages = sum(need) + spare
        self.rows = sum(n for n, _ in seqs)
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        self.pages = torch.full((len(seqs), max(need + [1])), -7, dtype=torch.int32, device=dev)
        at, start = 0, [0]
        self.codes, self.scales = {}, {}
        for name in "kv":
            self.codes[name] = torch.full((n_pages, H, P, D), 0xFF, dtype=torch.uint8, device=dev)
            self.scales[name] = torch.full((n_pages, H), float("nan"), device=dev)
        for i, (n, k) in enumerate(seqs):
            ids = order[at:at + need[i]]
            at += need[i]
            self.pages[i, :need[i]] = ids
            start.append(start[-1] + n)
            for name in "kv":
                c = torch.randint(0, 256, (need[i], H, P, D), generator=g, device=dev)
                c = torch.where((c & 127) == 127, c - 1, c)          # finite codes
                t = torch.arange(need[i] * P, device=dev).view(need[i], 1, P, 1)
                c = torch.where(t < k, c, torch.full_like(c, 0xFF)).to(torch.uint8)
                self.codes[name][ids.long()] = c
                e = torch.randint(-9, -5, (need[i], H), generator=g, device=dev)
                self.scales[name][ids.long()] = torch.exp2(e.float())
        self.row_start = torch.tensor(start, dtype=torch.int32, device=dev)
        self.kv_len = torch.tensor([k for _, k in seqs], dtype=torch.int32, device=dev)
        self.net = m.Attention(shape, max_rows=max_rows or max(self.rows, 1), max_seqs=len(seqs))
        self.cache = m.KVCache(self.codes["k"], self.codes["v"], self.scales["k"],
                               self.scales["v"])
        kw = dict(max_seq_rows=max(n for n, _ in seqs), max_kv_len=max(k for _, k in seqs)) \
            if hints is True else hints
        self.batch = m.AttnBatch(self.row_start, self.kv_len, self.pages, self.rows, **kw)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device=self.dev).to(torch.bfloat16)

    def q(self):
        return self.randn(self.rows, self.shape.q_heads, self.shape.head_dim)

    def expected(self, q):
        return R.attention(self.shape, q, self.codes["k"], self.scales["k"], self.codes["v"],
                           self.scales["v"], self.pages, self.row_start, self.kv_len)

    def check(self, q=None, out=None):
        q = self.q() if q is None else q
        out = self.net.forward(q, self.cache, self.batch, out=out)
        want, tol = self.expected(q)
        check_close(out, want, tol)
        assert self.net.device_status() == m.MOE_OK
        return out


def check_close(got, want, tol):
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    off = (got - want).abs()
    bad = (off > tol) & ~nan
    assert not bool(bad.any()), (int(bad.sum()), float((off / tol.clamp(min=1e-30))[~nan].max()))


# ---- rotary positions --------------------------------------------------------

@pytest.mark.parametrize("D,rot,layout,scaling,heads,rows,norm", [
    (128, 128, "half", "plain", 18, 1, False),
    (128, 32, "half", "plain", 18, 5, True),
    (128, 20, "half", "linear", 3, 33, True),          # half of the rotated part: 10 values
    (64, 2, "half", "plain", 1, 7, False),
    (64, 64, "interleaved", "by_parts", 9, 129, True),
    (256, 256, "half", "by_parts", 5, 40, False),
    (256, 250, "interleaved", "linear", 70, 3, True),
    (256, 6, "interleaved", "plain", 2, 300, False),
    (128, 0, "half", "plain", 4, 9, True)])
def test_rope(dev, D, rot, layout, scaling, heads, rows, norm):
    shape = m.AttnShape(q_heads=4, kv_heads=1, head_dim=D, rotary_dim=rot, rope_layout=layout,
                        rope_scaling=scaling, rope_factor=8.0, rope_trained_positions=4096,
                        rope_turns_low=1.0, rope_turns_high=32.0,
                        rope_amplitude=1.25 if scaling == "by_parts" else 1.0)
    g = gen(dev, rows)
    net = m.Attention(shape, max_rows=1)
    x = torch.randn((rows, heads, D), generator=g, device=dev).to(torch.bfloat16)
    gamma = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) if norm else None
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, device=dev).to(torch.int32)
    pos[0] = -5
    if rows > 2:
        pos[1], pos[2] = 0, 1 << 20
    y = net.rope(x, pos, gamma=gamma)
    want, tol = R.rope(shape, x, pos, gamma)
    check_close(y.cpu(), want, tol)
    # in place, and between rows of a wider tensor: the same bits
    z = x.clone()
    net.rope(z, pos, gamma=gamma, out=z)
    assert torch.equal(z.view(torch.int16), y.view(torch.int16))
    wide = torch.zeros((rows, heads + 3, D), dtype=torch.bfloat16, device=dev)
    wide[:, 1:1 + heads] = x
    out = torch.zeros((rows, heads + 1, D), dtype=torch.bfloat16, device=dev)
    net.rope(wide[:, 1:1 + heads], pos, gamma=gamma, out=out[:, :heads])
    assert torch.equal(out[:, :heads].contiguous().view(torch.int16), y.view(torch.int16))
    assert not bool(out[:, heads:].any())
    assert net.device_status() == m.MOE_OK


def test_rope_row_with_a_nan_stays_alone(dev):
    net = m.Attention(m.AttnShape(rotary_dim=64), max_rows=1)
    x = torch.randn((4, 3, 128), device=dev).to(torch.bfloat16)
    pos = torch.arange(4, dtype=torch.int32, device=dev)
    y = net.rope(x, pos)
    x[2, 1, 5] = float("nan")
    z = net.rope(x, pos)
    assert bool(torch.isnan(z[2, 1, 5])) and int(torch.isnan(z).sum()) == 2
    same = ~torch.isnan(z)
    assert torch.equal(z[same], y[same])


# ---- append --------------------------------------------------------------------

def appended(c, k, v):
    """The plain append of copies of the case's cache: {name: (codes, scales)}."""
    got = {}
    for name, x in (("k", k), ("v", v)):
        codes, scales = c.codes[name].cpu().clone(), c.scales[name].cpu().clone()
        R.append(c.shape, codes, scales, c.pages.cpu(), c.row_start.tolist(), c.kv_len.tolist(),
                 x.cpu())
        got[name] = (codes, scales)
    return got


def check_cache(c, want):
    for name in "kv":
        codes, scales = want[name]
        assert torch.equal(c.codes[name].cpu(), codes), name
        a, b = c.scales[name].cpu(), scales
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)), name


@pytest.mark.parametrize("D,P,H,seqs", [
    (128, 64, 2, [(1, 1)]), (128, 64, 2, [(1, 64)]), (128, 64, 2, [(1, 65)]),
    (64, 16, 3, [(1, 16), (0, 40), (1, 17), (5, 21)]),
    (128, 128, 1, [(200, 333), (1, 128), (129, 129)]),
    (256, 128, 2, [(127, 255), (0, 0), (128, 128)]),
    (256, 32, 1, [(70, 70), (3, 35)]),
    (64, 128, 5, [(1, 100), (300, 301)]),
    (128, 32, 2, [(10, 4), (3, 0), (2, 2)])])        # rows in front of the cache are not stored
def test_append(dev, D, P, H, seqs):
    shape = m.AttnShape(q_heads=H, kv_heads=H, head_dim=D, page_tokens=P, rotary_dim=0)
    c = Case(dev, shape, seqs, seed=D + P)
    size = torch.exp2(torch.randint(-6, 7, (c.rows, H, 1), generator=c.g, device=dev).float())
    k = (c.randn(c.rows, H, D) * size).to(torch.bfloat16)
    v = c.randn(c.rows, H, D)
    want = appended(c, k, v)
    c.net.append(k, v, c.cache, c.batch)
    check_cache(c, want)
    assert c.net.device_status() == m.MOE_OK


def test_append_token_by_token_keeps_normal_codes(dev):
    """One token a call: scales only grow, by powers of two, so codes that are not
    subnormal under the page's last scale are those of one call with all tokens."""
    shape = m.AttnShape(q_heads=2, kv_heads=2, head_dim=128, page_tokens=64, rotary_dim=0)
    n = 130
    one, all_ = Case(dev, shape, [(1, n)], seed=3), Case(dev, shape, [(n, n)], seed=3)
    k, v = all_.randn(n, 2, 128), all_.randn(n, 2, 128)
    k *= torch.exp2(torch.arange(n, device=dev) % 7 - 3.0)[:, None, None].to(torch.bfloat16)
    for t in range(n):
        one.kv_len.fill_(t + 1)
        one.net.append(k[t:t + 1], v[t:t + 1], one.cache, one.batch)
    all_.net.append(k, v, all_.cache, all_.batch)
    for name, x in (("k", k), ("v", v)):
        for j in range(3):
            a, b = int(one.pages[0, j]), int(all_.pages[0, j])
            t = min(64, n - 64 * j)
            assert torch.equal(one.scales[name][a], all_.scales[name][b])
            ca, cb = one.codes[name][a, :, :t], all_.codes[name][b, :, :t]
            normal = (cb & 0x78) != 0
            assert torch.equal(ca[normal], cb[normal])
            # subnormal codes: within one step
            off = ((ca & 127).int() - (cb & 127).int()).abs()
            assert not bool((off[~normal] > 1).any())


def test_append_nonfinite_rows_and_strided_inputs(dev):
    shape = m.AttnShape(q_heads=3, kv_heads=3, head_dim=64, page_tokens=16, rotary_dim=0)
    c = Case(dev, shape, [(9, 30), (20, 20)], seed=9)
    wide = c.randn(c.rows, 3 + 3 + 3, 64)
    k, v = wide[:, 3:6], wide[:, 6:]
    k[4, 1, 7], v[2, 0, 0], k[20, 2, 63] = float("nan"), float("inf"), float("-inf")
    k[12, 0] = 0
    want = appended(c, k, v)
    c.net.append(k, v, c.cache, c.batch)
    check_cache(c, want)


# ---- attention --------------------------------------------------------------------

SHAPES = [dict(q_heads=16, kv_heads=2, head_dim=128, page_tokens=64),
          dict(q_heads=6, kv_heads=2, head_dim=64, page_tokens=16),
          dict(q_heads=5, kv_heads=1, head_dim=256, page_tokens=32),
          dict(q_heads=16, kv_heads=1, head_dim=128, page_tokens=128),
          dict(q_heads=4, kv_heads=4, head_dim=64, page_tokens=128),
          dict(q_heads=7, kv_heads=1, head_dim=256, page_tokens=128)]


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("seqs", [
    [(1, 1)], [(1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 127), (1, 128), (1, 129)],
    [(1, 2000), (1, 3), (0, 50), (1, 700)],
    [(11, 11), (11, 300), (2, 2)],
    [(5, 3), (1, 0), (3, 1), (2, 90)]],               # rows that see no key
    ids=["one", "edges", "ragged", "frames", "empty"])
def test_attention_few_rows(dev, kw, seqs):
    c = Case(dev, m.AttnShape(rotary_dim=0, **kw), seqs, seed=len(seqs))
    q = c.q()
    out = c.check(q)
    for i, (n, k) in enumerate(seqs):                  # rows in front of the cache are zero
        r0 = int(c.row_start[i])
        for t in range(min(n, max(0, n - k))):
            assert not bool(out[r0 + t].any())


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("window", [1, 5, 64, 100])
def test_attention_window(dev, kw, window):
    c = Case(dev, m.AttnShape(rotary_dim=0, window=window, **kw),
             [(1, 200), (30, 90), (1, 5), (3, 64 + window), (140, 300)], seed=window)
    c.check()


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("seqs", [[(300, 300)], [(129, 500), (128, 128), (1, 77), (64, 64)],
                                  [(17, 1100), (260, 261)], [(200, 130), (90, 1000)]],
                         ids=["prompt", "ragged", "late", "empty"])
def test_attention_many_rows(dev, kw, seqs):
    Case(dev, m.AttnShape(rotary_dim=0, **kw), seqs, seed=7).check()


@pytest.mark.parametrize("seqs", [[(1, 20000)], [(40, 9000)], [(150, 6000)]])
def test_attention_long(dev, seqs):
    """Few rows over a long axis: many CTAs share a row tile."""
    c = Case(dev, m.AttnShape(q_heads=8, kv_heads=1, head_dim=128, page_tokens=64, rotary_dim=0),
             seqs, seed=11)
    q = c.q()
    a = c.check(q).clone()
    for _ in range(3):
        b = c.net.forward(q, c.cache, c.batch)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("D,rows", [(64, 12), (64, 20), (128, 21), (128, 31), (256, 45), (256, 60)])
@pytest.mark.parametrize("window", [0, 130])
def test_attention_few_row_tiles(dev, D, rows, window):
    """Tiles of 16 rows (three tokens of five heads) up to the number at which the prompt
    kernel takes over, and the one behind it, with keys shared out either way."""
    shape = m.AttnShape(q_heads=5, kv_heads=1, head_dim=D, page_tokens=32, rotary_dim=0,
                        window=window)
    for ctx in (rows, rows + 1, 1000):
        Case(dev, shape, [(rows, ctx)], seed=rows + ctx).check()


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [40, 150])
def test_attention_long_other_widths(dev, D, rows):
    """More parts of a row block than one thread joins, at the other head widths."""
    shape = m.AttnShape(q_heads=14, kv_heads=2, head_dim=D, page_tokens=128, rotary_dim=0)
    Case(dev, shape, [(rows, 7000)], seed=D + rows).check()


@pytest.mark.parametrize("n,most", [(40, 100), (130, 1000), (300, 30), (700, 900), (4000, 40)])
def test_attention_many_sequences(dev, n, most):
    """A row of each of many sequences, lengths from none to `most`: as runs of key tiles and
    as a CTA to each, whichever the sizes call for."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, most + 1, (n,), generator=g).tolist()
    shape = m.AttnShape(q_heads=4, kv_heads=2, head_dim=64, page_tokens=16, rotary_dim=0)
    Case(dev, shape, [(1, k) for k in lens], seed=n).check()


@pytest.mark.parametrize("window", [300, 0x7FFEFFFF, 0x7FFFFFFF])
def test_attention_windows_past_all_tokens(dev, window):
    """A window wider than the cache sees what no window sees, bit for bit."""
    kw = dict(q_heads=4, kv_heads=2, head_dim=128, page_tokens=64, rotary_dim=0)
    for seqs in ([(1, 200), (3, 2)], [(200, 290)]):
        a = Case(dev, m.AttnShape(**kw), seqs, seed=3)
        b = Case(dev, m.AttnShape(window=window, **kw), seqs, seed=3)
        q = a.q()
        x, y = a.check(q), b.check(q)
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("hints", [dict(), dict(max_seq_rows=1, max_kv_len=1),
                                   dict(max_seq_rows=60000, max_kv_len=1 << 30)])
def test_attention_hints_only_size_the_launch(dev, hints):
    c = Case(dev, m.AttnShape(q_heads=4, kv_heads=2, head_dim=64, page_tokens=32, rotary_dim=0),
             [(1, 300), (70, 150), (200, 1000)], seed=2, hints=hints)
    c.check()


def test_attention_scores_far_apart(dev):
    """Queries of very unlike sizes: scores from nearly equal to hundreds apart, one key that
    takes everything, and a softmax scale of the caller's."""
    shape = m.AttnShape(q_heads=8, kv_heads=2, head_dim=128, page_tokens=64, rotary_dim=0,
                        softmax_scale=0.7)
    for seqs in ([(4, 500)], [(200, 500)]):
        c = Case(dev, shape, seqs, seed=5)
        size = torch.exp2(torch.randint(-20, 5, (c.rows, 8, 1), generator=c.g, device=dev).float())
        c.check((c.randn(c.rows, 8, 128) * size).to(torch.bfloat16))
        q = c.q()
        q[:, 3] = 0
        c.check(q)


@pytest.mark.parametrize("rows", [3, 150])
def test_attention_page_scales_of_any_size(dev, rows):
    """Scales that differ by 2^40 between pages, and ones that are no powers of two."""
    shape = m.AttnShape(q_heads=4, kv_heads=2, head_dim=128, page_tokens=16, rotary_dim=0)
    c = Case(dev, shape, [(rows, 400)], seed=8)
    n = c.scales["v"].shape
    c.scales["v"].copy_(torch.exp2(torch.randint(-30, 10, n, generator=c.g, device=dev).float()))
    c.check()
    c.scales["v"].copy_(0.001 + torch.rand(n, generator=c.g, device=dev))
    c.scales["k"].copy_(0.001 + 0.01 * torch.rand(n, generator=c.g, device=dev))
    c.check()


@pytest.mark.parametrize("rows", [6, 150])
@pytest.mark.parametrize("window", [0, 20])
def test_attention_nan_reaches_only_rows_that_see_it(dev, rows, window):
    shape = m.AttnShape(q_heads=4, kv_heads=2, head_dim=128, page_tokens=64, rotary_dim=0,
                        window=window)
    c = Case(dev, shape, [(rows, 300)], seed=4)
    page, slot = int(c.pages[0, 298 // 64]), 298 % 64       # seen by the last two rows
    c.codes["v"][page, 0, slot] = 0x7F
    old = int(c.pages[0, 3])                                # token 200: seen by all, or by none
    c.codes["k"][old, 1, 200 - 192, 5] = 0xFF
    q = c.q()
    q[1, 0, 3] = float("inf")                               # one head of one row
    q[2, 3, 100] = float("nan")
    out = c.net.forward(q, c.cache, c.batch)
    want, tol = c.expected(q)
    # heads 0, 1 read key head 0; a NaN value makes every value of a row that sees it NaN
    want[1, 0] = float("nan")
    want[2, 3] = float("nan")
    check_close(out, want, tol)
    first = 300 - rows
    for i in range(rows):
        sees = first + i >= 298
        assert bool(torch.isnan(out[i, 1]).all()) == sees
        k_seen = first + i >= 200 and (not window or 200 > first + i - window)
        assert bool(torch.isnan(out[i, 2]).all()) == k_seen


def test_attention_strided_rows_and_another_stream(dev):
    shape = m.AttnShape(q_heads=6, kv_heads=3, head_dim=64, page_tokens=32, rotary_dim=0)
    c = Case(dev, shape, [(1, 700), (9, 40), (1, 90)], seed=6)
    q = c.q()
    want = c.check(q)
    wide = torch.zeros((c.rows, 11, 64), dtype=torch.bfloat16, device=dev)
    wide[:, 2:8] = q
    out = torch.zeros((c.rows, 9, 64), dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.net.forward(wide[:, 2:8], c.cache, c.batch, out=out[:, 1:7], stream=side)
    side.synchronize()
    assert torch.equal(out[:, 1:7].contiguous().view(torch.int16), want.view(torch.int16))
    assert not bool(out[:, 0].any()) and not bool(out[:, 7:].any())


def test_attention_in_a_graph_with_growing_lengths(dev):
    shape = m.AttnShape(q_heads=8, kv_heads=2, head_dim=128, page_tokens=64)
    c = Case(dev, shape, [(1, 900), (1, 800)], seed=12)
    qkv = c.randn(2, 12, 128)
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device=dev)
    c.kv_len.fill_(1)
    c.net.step(qkv, c.cache, c.batch, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.net.step(qkv, c.cache, c.batch, out=out)
    for n in (5, 64, 65, 500, 900):
        c.kv_len.copy_(torch.tensor([n, max(1, n - 100)], dtype=torch.int32))
        graph.replay()
        a = out.clone()
        c.net.step(qkv, c.cache, c.batch, out=out)
        assert torch.equal(a.view(torch.int16), out.view(torch.int16)), n
    assert c.net.device_status() == m.MOE_OK


def test_attention_pages_behind_4_gib(dev):
    """Pages whose byte offsets pass 32 bits."""
    shape = m.AttnShape(q_heads=4, kv_heads=4, head_dim=256, page_tokens=128, rotary_dim=0)
    n_pages = (1 << 32) // (4 * 128 * 256) + 40
    codes = [torch.zeros((n_pages, 4, 128, 256), dtype=torch.uint8, device=dev) for _ in "kv"]
    scales = [torch.ones((n_pages, 4), device=dev) for _ in "kv"]
    cache = m.KVCache(*codes, *scales)
    for rows in (2, 300):
        small = Case(dev, shape, [(rows, 700)], seed=13)
        far = small.pages + (n_pages - small.codes["k"].shape[0])
        for big, name in zip(codes, "kv"):
            big[-small.codes[name].shape[0]:] = small.codes[name]
        for big, name in zip(scales, "kv"):
            big[-small.scales[name].shape[0]:] = small.scales[name]
        batch = m.AttnBatch(small.row_start, small.kv_len, far.contiguous(), rows, rows, 700)
        k, v, q = small.randn(rows, 4, 256), small.randn(rows, 4, 256), small.q()
        small.net.append(k, v, cache, batch)
        a = small.net.forward(q, cache, batch)
        small.net.append(k, v, small.cache, small.batch)
        b = small.net.forward(q, small.cache, small.batch)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        check_close(b, *small.expected(q))


# ---- the step ----------------------------------------------------------------------

@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kw,seqs", [
    (dict(q_heads=16, kv_heads=2, head_dim=128, page_tokens=64, rotary_dim=32),
     [(1, 900), (1, 1), (1, 65)]),
    (dict(q_heads=6, kv_heads=2, head_dim=64, page_tokens=16, rotary_dim=64,
          rope_layout="interleaved"), [(11, 200), (0, 3), (200, 200)]),
    (dict(q_heads=5, kv_heads=1, head_dim=256, page_tokens=128, rotary_dim=20, window=70),
     [(150, 400), (2, 2)])])
def test_step_is_its_parts(dev, kw, seqs, norm):
    """moe_attn_step: bit for bit moe_rope, moe_kv_append and moe_attn_forward."""
    shape = m.AttnShape(**kw)
    a, b = Case(dev, shape, seqs, seed=21), Case(dev, shape, seqs, seed=21)
    hq, hk, D = shape.q_heads, shape.kv_heads, shape.head_dim
    qkv = a.randn(a.rows, hq + 2 * hk, D)
    qg, kg = ((1 + 0.1 * a.randn(D)).to(torch.bfloat16) for _ in "qk") if norm else (None, None)
    out = a.net.step(qkv, a.cache, a.batch, q_gamma=qg, k_gamma=kg)
    pos = torch.cat([torch.arange(k - n, k) for n, k in seqs]).to(torch.int32).to(dev)
    q = b.net.rope(qkv[:, :hq], pos, gamma=qg)
    k = b.net.rope(qkv[:, hq:hq + hk], pos, gamma=kg)
    b.net.append(k, qkv[:, hq + hk:], b.cache, b.batch)
    want = b.net.forward(q, b.cache, b.batch)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    for name in "kv":
        assert torch.equal(a.codes[name], b.codes[name])
        assert torch.equal(torch.nan_to_num(a.scales[name]), torch.nan_to_num(b.scales[name]))
    check_close(out, *b.expected(q))
    assert a.net.device_status() == m.MOE_OK


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_step_of_one_head_rotated_whole(dev, D, layout):
    """One query head: a block of the prologue holds the sines of as many rows as it can."""
    shape = m.AttnShape(q_heads=1, kv_heads=1, head_dim=D, page_tokens=32, rotary_dim=D,
                        rope_layout=layout)
    for seqs in ([(1, 40)], [(130, 150), (70, 400), (1, 1)]):
        a, b = Case(dev, shape, seqs, seed=41), Case(dev, shape, seqs, seed=41)
        qkv = a.randn(a.rows, 3, D)
        out = a.net.step(qkv, a.cache, a.batch)
        pos = torch.cat([torch.arange(k - n, k) for n, k in seqs]).to(torch.int32).to(dev)
        q, k = b.net.rope(qkv[:, :1], pos), b.net.rope(qkv[:, 1:2], pos)
        b.net.append(k, qkv[:, 2:], b.cache, b.batch)
        assert torch.equal(a.codes["k"], b.codes["k"])
        check_close(out, *b.expected(q))
        assert a.net.device_status() == m.MOE_OK


# ---- refusals ----------------------------------------------------------------------

def test_refusals(dev):
    shape = m.AttnShape(q_heads=4, kv_heads=2, head_dim=64, page_tokens=16, rotary_dim=64)
    c = Case(dev, shape, [(2, 30)], max_rows=4)
    q, out = c.q(), torch.empty_like(c.q())
    ctx, bad = c.net.ctx, m.MOE_ERR_INVALID_ARG
    cc, bb = c.cache._c, c.batch._c

    def fwd(q=q, qs=256, out=out, os=256, cache=cc, batch=bb):
        return m.moe_attn_forward(ctx, cache, q, qs, batch, out, os)
    assert fwd() == m.MOE_OK
    assert fwd(q=None) == bad and fwd(out=None) == bad and fwd(cache=None) == bad
    assert fwd(batch=None) == bad and fwd(qs=248) == bad and fwd(os=260) == bad
    assert fwd(out=q) == bad and fwd(q=q.data_ptr() + 2) == bad

    def batch(**kw):
        b = m.moe_attn_batch(*[getattr(bb, n) for n, _ in m.moe_attn_batch._fields_])
        for k, v in kw.items():
            setattr(b, k, v)
        return b
    assert fwd(batch=batch(rows=5)) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert fwd(batch=batch(n_seqs=2)) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert fwd(batch=batch(rows=-1)) == bad and fwd(batch=batch(n_seqs=0)) == bad
    assert fwd(batch=batch(pages_stride=0)) == bad and fwd(batch=batch(pages=None)) == bad
    assert fwd(batch=batch(max_kv_len=-1)) == bad
    assert fwd(batch=batch(rows=0)) == m.MOE_OK
    pool = m.moe_kv_cache(cc.k_codes + 4, cc.v_codes, cc.k_scales, cc.v_scales, cc.n_pages)
    assert fwd(cache=pool) == bad
    pool = m.moe_kv_cache(cc.k_codes, cc.v_codes, cc.k_scales, cc.v_scales, 0)
    assert fwd(cache=pool) == bad
    pos = torch.zeros(2, dtype=torch.int32, device=dev)
    assert m.moe_rope(ctx, q, 256, 4, pos, None, -1.0, 2, out, 256) == bad
    assert m.moe_rope(ctx, q, 256, 4, pos, None, float("nan"), 2, out, 256) == bad
    assert m.moe_rope(ctx, q, 256, 0, pos, None, 0.0, 2, out, 256) == bad
    assert m.moe_rope(ctx, q, 256, 1025, pos, None, 0.0, 2, out, 256) == \
        m.MOE_ERR_UNSUPPORTED_SHAPE
    assert m.moe_rope(ctx, q, 256, 4, None, None, 0.0, 2, out, 256) == bad
    assert m.moe_rope(ctx, q, 256, 4, pos, None, 0.0, 2, q.data_ptr() + 16, 256) == bad
    assert m.moe_rope(ctx, None, 0, 4, None, None, 0.0, 0, None, 0) == m.MOE_OK
    assert m.moe_kv_append(ctx, cc, q, 120, q, 128, bb) == bad
    assert m.moe_attn_step(ctx, cc, q, 256, None, None, 1e-6, bb, out, 256) == bad
    with pytest.raises(ValueError):
        c.net.forward(q.float(), c.cache, c.batch)
    with pytest.raises(ValueError):
        c.net.forward(q[:1], c.cache, c.batch)
    with pytest.raises(ValueError):
        c.net.append(q, q, c.cache, c.batch)
    with pytest.raises(ValueError):
        m.AttnBatch(c.row_start.long(), c.kv_len, c.pages, 2)
    with pytest.raises(ValueError):
        m.KVCache(c.codes["k"], c.codes["v"][:, :1], c.scales["k"], c.scales["v"])
    torch.cuda.synchronize()
    assert c.net.device_status() == m.MOE_OK


@pytest.mark.parametrize("rows", [1, 200])
def test_batches_out_of_range_are_reported_not_followed(dev, rows):
    """Page numbers, lengths and row starts out of range: nothing outside the buffers is
    touched, the status says so, other sequences are right, and the next call is."""
    shape = m.AttnShape(q_heads=4, kv_heads=2, head_dim=64, page_tokens=16, rotary_dim=0)
    c = Case(dev, shape, [(1, 50), (rows, 300), (2, 40)], seed=31)
    q = c.q()
    good = c.check(q).clone()
    keep = {n: getattr(c, n).clone() for n in ("pages", "kv_len", "row_start")}
    k = c.randn(c.rows, 2, 64)

    def spoil(name, at, value, intact):
        getattr(c, name)[at] = value
        out = c.net.forward(q, c.cache, c.batch)
        assert c.net.device_status() == m.MOE_ERR_INVALID_ARG
        assert torch.equal(out[intact].view(torch.int16), good[intact].view(torch.int16))
        getattr(c, name).copy_(keep[name])
        assert c.net.device_status() == m.MOE_OK
        c.check(q)
    others = torch.tensor([0, 1 + rows, 2 + rows], device=dev)
    spoil("pages", (1, 2), -1, others)
    spoil("pages", (1, 18), c.codes["k"].shape[0], others)
    spoil("pages", (1, 0), 2 ** 31 - 1, others)
    spoil("kv_len", 1, -3, others)
    spoil("kv_len", 1, 2 ** 31 - 1, others[:1])
    spoil("row_start", 3, 2 ** 30, torch.tensor([0], device=dev))
    # an append to a page that does not exist stores nothing
    c.pages[0, 3] = -1
    before = c.codes["k"].clone()
    c.kv_len[1:] = 0
    c.net.append(k, k, c.cache, c.batch)
    assert c.net.device_status() == m.MOE_ERR_INVALID_ARG
    assert torch.equal(c.codes["k"], before)
