"""Rows to their experts and back on the GPU against the plain 64-bit forms
(tests/ops_reference.py): orders, dropped pairs, ragged widths, strides (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

import ops_reference as R

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


def experts(dev, tokens, k, n, kind, seed=0):
    g = gen(dev, seed)
    if kind == "distinct" and k <= n:
        return torch.rand((tokens, n), generator=g, device=dev).argsort(1)[:, :k].to(torch.int32)
    idx = torch.randint(0, n, (tokens, k), generator=g, device=dev, dtype=torch.int32)
    if kind == "one":                      # every pair to one expert
        return torch.full_like(idx, n - 1)
    if kind == "none":
        return torch.full_like(idx, -1)
    if kind == "dropped":
        bad = torch.tensor([-1, n, -2 ** 31, 2 ** 31 - 1], device=dev, dtype=torch.int32)
        pick = bad[torch.randint(0, 4, (tokens, k), generator=g, device=dev)]
        idx = torch.where(torch.rand((tokens, k), generator=g, device=dev) < 0.4, pick, idx)
        idx[tokens // 2] = -1              # a token without any row
    return idx                             # "any": the same expert twice in a token, too


def sentinel(rows, width, dev, quantize, ops):
    if quantize:
        return m.QuantRows(torch.full((rows, width), 0xA5, dtype=torch.uint8, device=dev),
                           torch.full((rows, -(-width // 128)), -3.0, device=dev))
    return torch.full((rows, width), -77.0, dtype=torch.bfloat16, device=dev)


CASES = [  # tokens, top_k, experts, width, kind
    (1, 8, 256, 2048, "distinct"), (1, 1, 1, 16, "any"), (11, 8, 256, 2048, "distinct"),
    (3, 16, 4, 128, "any"), (153, 8, 256, 272, "dropped"), (700, 6, 60, 1040, "any"),
    (200, 5, 7, 2560, "one"), (64, 2, 3, 144, "none"), (1536, 8, 256, 48, "any"),
    (1537, 8, 256, 80, "dropped"), (2048, 8, 256, 48, "any"),
    (2049, 8, 256, 64, "dropped"), (5000, 7, 100, 128, "any"), (20000, 1, 5, 16, "dropped"),
    (9001, 16, 256, 32, "one"), (65536, 16, 256, 16, "any")]


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_dispatch(dev, case, quantize):
    tokens, k, n, width, kind = case
    idx = experts(dev, tokens, k, n, kind)
    x = (torch.randn((tokens, width), generator=gen(dev, 1), device=dev)
         * torch.exp(2 * torch.randn((tokens, 1), generator=gen(dev, 2), device=dev))).bfloat16()
    ops = m.ExpertOps(n, k, tokens, 0)
    out = sentinel(tokens * k, width, dev, quantize, ops)
    order, got = ops.dispatch(x, idx, out=out)
    starts, pair, slot = R.order(idx, n)
    assert torch.equal(order.starts, starts)
    assert torch.equal(order.pair_of_slot, pair)
    assert torch.equal(order.slot_of_pair, slot)
    kept = int(starts[-1])
    token = pair[:kept].long() // k
    if quantize:
        codes, scales = R.quantise(x)
        want = sentinel(tokens * k, width, dev, True, ops)
        want.codes[:kept], want.scales[:kept] = codes[token], scales[token]
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    else:
        want = sentinel(tokens * k, width, dev, False, ops)
        want[:kept] = x[token]
        assert torch.equal(got, want)
    assert torch.equal(ops.sort(idx).slot_of_pair, slot)   # the order alone
    assert ops.device_status() == m.MOE_OK


@pytest.mark.parametrize("case", CASES + [(5, 8, 16, 8, "any"), (70, 3, 16, 2056, "dropped")],
                         ids=str)
def test_combine_and_gradients(dev, case):
    tokens, k, n, width, kind = case
    idx = experts(dev, tokens, k, n, kind)
    ops = m.ExpertOps(n, k, tokens, 0)
    order = ops.sort(idx)
    kept, slot, pairs = int(order.starts[-1]), order.slot_of_pair, tokens * k
    g = gen(dev, 5)
    rows = torch.randn((pairs, width), generator=g, device=dev).bfloat16()
    rows[kept:] = float("nan")             # rows of no pair are not read
    w = torch.randn((tokens, k), generator=g, device=dev)
    w[slot < 0] = float("nan")             # nor weights of pairs without a row
    dy = torch.randn((tokens, width), generator=g, device=dev).bfloat16()

    # k products and k sums in fp32, one rounding to bf16
    want, mag = R.combine(rows, slot, w)
    err = (ops.combine(rows, order, w).double() - want).abs()
    assert bool((err <= BOUND(k) * mag + R.BF16 * (1 + 2.0 ** -7) * want.abs()).all())
    want, mag = R.combine(rows, slot)
    err = (ops.dispatch_grad(rows, order).double() - want).abs()
    assert bool((err <= BOUND(k) * mag + R.BF16 * (1 + 2.0 ** -7) * want.abs()).all())

    out = sentinel(pairs, width, dev, False, ops)
    out, dw = ops.combine_grad(dy, rows, order, w, out=out)
    pair = order.pair_of_slot[:kept].long()
    product = w.flatten()[pair][:, None] * dy[pair // k].float()
    want = sentinel(pairs, width, dev, False, ops)
    want[:kept] = product.bfloat16()
    assert torch.equal(out, want)
    terms = dy[pair // k].double() * rows[:kept].double()
    want = torch.zeros(pairs, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(want)
    want[pair], mag[pair] = terms.sum(1), terms.abs().sum(1)
    # a lane's products one after the other, then five sums of lanes
    err = (dw.flatten().double() - want).abs()
    assert bool((err <= (width / 32 + 24) * 2.0 ** -24 * mag).all())
    if width % 16 == 0:
        got, dw2 = ops.combine_grad(dy, rows, order, w, out=sentinel(pairs, width, dev, True, ops))
        codes, scales = R.quantise(product)
        want = sentinel(pairs, width, dev, True, ops)
        want.codes[:kept], want.scales[:kept] = codes, scales
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
        assert torch.equal(dw, dw2)
    assert ops.device_status() == m.MOE_OK


def BOUND(k):
    return (2 * k + 1) * 2.0 ** -24


def test_gradients_are_the_derivatives():
    """The gradients' formulas against autograd and against differences, in 64 bits."""
    torch.manual_seed(0)
    idx = torch.tensor([[0, 2], [1, 1], [-1, 0], [5, -1]], dtype=torch.int32)
    starts, pair, slot = R.order(idx, 3)
    x = torch.randn(4, 3, dtype=torch.float64, requires_grad=True)
    rows = torch.randn(8, 3, dtype=torch.float64, requires_grad=True)
    w = torch.randn(4, 2, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(4, 3, dtype=torch.float64)

    def forward(rows, w):
        there = (slot >= 0)[..., None]
        return ((rows[slot.clamp(min=0).long()] * w[..., None]) * there).sum(1)
    drows, dw = torch.autograd.grad((forward(rows, w) * dy).sum(), (rows, w))
    kept = int(starts[-1])
    at = pair[:kept].long()
    assert torch.allclose(drows[:kept], w.flatten()[at][:, None] * dy[at // 2])
    assert bool((drows[kept:] == 0).all())
    for t in range(4):
        for j in range(2):
            e = torch.zeros_like(w)
            e[t, j] = 1e-6
            d = ((forward(rows, w + e) - forward(rows, w - e)) * dy).sum() / 2e-6
            s = int(slot[t, j])
            want = float(dy[t] @ rows[s]) if s >= 0 else 0.0
            assert abs(float(d) - want) < 1e-6 and abs(float(dw[t, j]) - want) < 1e-12
    # dispatch: rows = x[token]; its gradient is the unweighted sum
    drows = torch.randn(8, 3, dtype=torch.float64)
    dx, = torch.autograd.grad((x[at // 2] * drows[:kept]).sum(), x)
    assert torch.allclose(dx, R.combine(drows, slot)[0])


def test_order_needs_no_row_and_no_token(dev):
    ops = m.ExpertOps(16, 2, 8, 128)
    order, rows = ops.dispatch(torch.empty((0, 64), dtype=torch.bfloat16, device=dev),
                               torch.empty((0, 2), dtype=torch.int32, device=dev))
    assert order.tokens == 0 and rows.shape == (0, 64) and order.starts.sum() == 0
    assert ops.combine(rows, order, torch.empty((0, 2), device=dev)).shape == (0, 64)


def test_strides(dev):
    """Rows that are columns of wider buffers; what lies between them stays."""
    tokens, k, n, width = 37, 3, 9, 80
    ops = m.ExpertOps(n, k, tokens, 0)
    idx = experts(dev, tokens, k, n, "dropped")
    wide = torch.randn((tokens, 200), generator=gen(dev, 3), device=dev).bfloat16()
    x = wide[:, 16:16 + width]
    buf = torch.full((tokens * k, 128), 5.0, dtype=torch.bfloat16, device=dev)
    order, rows = ops.dispatch(x, idx, out=buf[:, 8:8 + width])
    plain = ops.dispatch(x.contiguous(), idx)[1]
    kept = int(order.starts[-1])
    assert torch.equal(rows[:kept], plain[:kept])
    assert bool((buf[:, :8] == 5).all()) and bool((buf[:, 88:] == 5).all())
    assert bool((buf[kept:] == 5).all())
    w = torch.rand((tokens, k), generator=gen(dev, 4), device=dev)
    y = torch.full((tokens, 104), 6.0, dtype=torch.bfloat16, device=dev)
    ops.combine(rows, order, w, out=y[:, 24:])
    assert torch.equal(y[:, 24:], ops.combine(rows.contiguous(), order, w))
    assert bool((y[:, :24] == 6).all())
    d = torch.full((tokens * k, 96), 7.0, dtype=torch.bfloat16, device=dev)
    _, dw = ops.combine_grad(y[:, 24:], rows, order, w, out=d[:, :width])
    ref, dw2 = ops.combine_grad(y[:, 24:].contiguous(), rows.contiguous(), order, w)
    assert torch.equal(d[:kept, :width], ref[:kept]) and torch.equal(dw, dw2)
    assert bool((d[:, width:] == 7).all()) and bool((d[kept:] == 7).all())


def test_infinities_and_nans_stay_in_their_rows(dev):
    tokens, k, n, width = 12, 2, 5, 256
    ops = m.ExpertOps(n, k, tokens, 0)
    idx = experts(dev, tokens, k, n, "any")
    x = torch.randn((tokens, width), generator=gen(dev, 6), device=dev).bfloat16()
    clean = ops.dispatch(x, idx, quantize=True)[1]
    x[3, 7], x[5, 200] = float("inf"), float("nan")
    order, got = ops.dispatch(x, idx, quantize=True)
    token = order.pair_of_slot.long() // k
    v = R.values(got.codes, got.scales)
    for row in range(tokens * k):
        t = int(token[row])
        if t not in (3, 5):
            assert torch.equal(got.codes[row], clean.codes[row])
        elif t == 3:
            assert not bool(torch.isfinite(v[row, :128]).all())
            assert bool(torch.isfinite(v[row, 128:]).all())
        else:
            assert bool(v[row, 200].isnan())


def test_codes_at_the_ends_of_the_range(dev):
    """Groups from bf16's smallest subnormal to its largest value, zeros among them, and rows
    whose product with a weight is tiny or huge: codes and scales bit for bit."""
    g = gen(dev, 8)
    e = torch.tensor([-133, -130, -126, -110, -90, -81, -80, -79, -40, 0, 60, 99, 100, 101, 120,
                      127], device=dev)
    tokens, width = len(e) * 3, 400
    x = torch.randn((tokens, width), generator=g, device=dev).clamp(-1.9, 1.9)
    x = (x.double() * torch.exp2(e.double()).repeat(3)[:, None]).bfloat16()
    x[::5, 128:256] = 0.0
    x[1::7, ::3] = 0.0
    x[2::7, 5] = -0.0
    idx = torch.arange(tokens, device=dev, dtype=torch.int32)[:, None] % 7
    ops = m.ExpertOps(7, 1, tokens, 0)
    order, got = ops.dispatch(x, idx.contiguous(), quantize=True)
    codes, scales = R.quantise(x)
    at = order.pair_of_slot.long()
    assert torch.equal(got.codes, codes[at]) and torch.equal(got.scales, scales[at])
    for weight in (1.0, 2.0 ** -30 / 3, 0.0, -2.0 ** 20 / 3):
        w = torch.full((tokens, 1), weight, device=dev)
        out, _ = ops.combine_grad(x, x[at].contiguous(), order, w, quantize=True)
        codes, scales = R.quantise((w * x.float())[at])
        assert torch.equal(out.scales, scales) and torch.equal(out.codes, codes)


def test_columns_of_one_buffer(dev):
    """Token rows and their pairs' rows as columns of one buffer; sharing a byte is refused."""
    tokens, k = 6, 3
    ops = m.ExpertOps(4, k, tokens, 0)
    idx = experts(dev, tokens, k, 4, "any")
    buf = torch.zeros((tokens * k, 64), dtype=torch.bfloat16, device=dev)
    buf[:tokens, :16] = torch.randn((tokens, 16), generator=gen(dev, 9), device=dev).bfloat16()
    order, rows = ops.dispatch(buf[:tokens, :16], idx, out=buf[:, 16:32])
    assert torch.equal(rows, buf[:tokens, :16][order.pair_of_slot.long() // k])
    ops.combine(rows, order, torch.ones((tokens, k), device=dev), out=buf[:tokens, 32:48])
    for out in (buf[:, 8:24], buf[:, :16]):
        with pytest.raises(m.MoEError) as e:
            ops.dispatch(buf[tokens:2 * tokens, :16], idx, out=out)
        assert e.value.status == m.MOE_ERR_INVALID_ARG


def test_long_offsets(dev):
    """Rows whose offsets pass 2^31 values."""
    tokens, k, width = 65536, 9, 4096
    ops = m.ExpertOps(2, k, tokens, 0)
    idx = torch.ones((tokens, k), dtype=torch.int32, device=dev)
    x = (torch.arange(tokens, device=dev) % 251).bfloat16()[:, None].repeat(1, width)
    order, rows = ops.dispatch(x, idx)
    assert rows.numel() > 2 ** 31
    at = torch.tensor([0, 524287, 524288, 589823], device=dev)
    assert torch.equal(rows[at], x[at // k])
    w = torch.zeros((tokens, k), device=dev)
    w[:, k - 1] = 2.0
    y = ops.combine(rows, order, w)
    assert torch.equal(y, 2 * x)
    out, dw = ops.combine_grad(x, rows, order, w, out=torch.empty_like(rows))
    assert torch.equal(out[at[3]], 2 * x[-1]) and bool((out[at[2]] == 0).any())
    assert float(dw[-1, 0]) == float(x[-1].double().square().sum())
