"""The block-FP8 product and its gradient on the GPU against the plain 64-bit form
(tests/ops_reference.py): ragged groups, odd sizes, strides, both forms of rows (needs a
GB300)."""
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


def weights(dev, groups, out, inner, seed=0):
    g = gen(dev, seed)
    c = torch.randint(0, 256, (groups, out, inner), generator=g, device=dev, dtype=torch.int32)
    c = torch.where((c & 127) == 127, c - 1, c).to(torch.uint8)        # finite codes
    s = torch.exp2(3 * torch.rand((groups, -(-out // 128), -(-inner // 128)), generator=g,
                                  device=dev) - 9)
    return m.BlockWeights(c, s)


def starts_of(counts, dev):
    return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32,
                        device=dev)


def bound(inner):
    """Error of the fp32 sums, relative to the sum of magnitudes.  A block's 128 products are
    exact and added with at most one part in 2^23 lost an addition; a block's product, its
    scale and the sum over the blocks are rounded to fp32."""
    return (128 + 4 + -(-inner // 128)) * 2.0 ** -23


def check(dev, counts, out, inner, trans, quantized, rows=None, seed=0):
    w = weights(dev, len(counts), out, inner, seed)
    starts = starts_of(counts, dev)
    rows = sum(counts) if rows is None else rows
    K, N = (out, inner) if trans else (inner, out)
    x = (torch.randn((rows, K), generator=gen(dev, seed + 1), device=dev) *
         torch.exp(torch.randn((rows, 1), generator=gen(dev, seed + 2), device=dev))).bfloat16()
    codes, scales = R.quantise(x)
    ops = m.ExpertOps(1, 1, max(rows, 1), 0 if quantized else K)
    y = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device=dev)
    (ops.linear_grad if trans else ops.linear)(m.QuantRows(codes, scales) if quantized else x, w,
                                               starts=starts, out=y)
    keep = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device=dev)
    want, mag = R.linear(R.values(codes, scales), w.codes, w.scales, starts.tolist(), keep, trans)
    err = (y.double() - want).abs()
    assert bool((err <= bound(K) * mag + R.BF16 * (1 + 2.0 ** -7) * want.abs()).all()), \
        float((err / (bound(K) * mag + R.BF16 * want.abs() + 1e-30)).max())
    assert torch.equal(y[sum(counts):], keep[sum(counts):])
    assert ops.device_status() == m.MOE_OK


GROUPS = [  # rows of each group
    [1], [5], [8], [9], [33], [64], [65], [128], [129], [300], [1000],
    [0, 3, 0, 128, 1, 129, 0], [7] * 40, [1] * 88, [0] * 255 + [2], [700, 1, 0, 90]]
SIZES = [(256, 256), (128, 128), (16, 16), (48, 400), (2560, 2048), (272, 1040), (384, 144),
         (1024, 528)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_one_group(dev, size, trans):
    for n, quantized in ((1, False), (3, True), (40, False), (200, True)):
        check(dev, [n], *size, trans, quantized)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_groups(dev, counts, trans):
    check(dev, counts, 400, 272, trans, True)
    check(dev, counts, 512, 640, trans, False, rows=sum(counts) + 13)
    # few rows of weights this large are few rows to the one kernel, many to the other
    check(dev, counts, 1552, 1808, trans, len(counts) % 2 == 0)


def test_many_tiles(dev):
    """More tiles than SMs, many blocks of the contraction."""
    check(dev, [777, 0, 3000, 130, 1], 1360, 4096, False, True)
    check(dev, [777, 0, 3000, 130, 1], 4096, 1360, True, False)


def test_no_rows(dev):
    w = weights(dev, 4, 128, 256)
    ops = m.ExpertOps(4, 2, 8, 256)
    starts = torch.zeros(5, dtype=torch.int32, device=dev)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=dev)
    assert ops.linear(x, w, starts=starts).shape == (0, 128)
    x = torch.ones((6, 256), dtype=torch.bfloat16, device=dev)
    y = torch.full((6, 128), 3.0, dtype=torch.bfloat16, device=dev)
    ops.linear(x, w, starts=starts, out=y)          # every group empty
    assert bool((y == 3).all()) and ops.device_status() == m.MOE_OK


def test_dense_without_starts(dev):
    w = weights(dev, 1, 384, 256)
    ops = m.ExpertOps(1, 1, 100, 256)
    x = torch.randn((100, 256), generator=gen(dev, 1), device=dev).bfloat16()
    a = ops.linear(x, w)
    assert torch.equal(a, ops.linear(x, w, starts=starts_of([100], dev)))
    assert torch.equal(a, ops.linear(x, m.BlockWeights(w.codes[0], w.scales[0])))


@pytest.mark.parametrize("rows", [1, 4, 20, 200])
def test_strides(dev, rows):
    w = weights(dev, 1, 272, 256)
    ops = m.ExpertOps(1, 1, rows, 272)
    wide = torch.randn((rows, 400), generator=gen(dev, 1), device=dev).bfloat16()
    x = wide[:, 8:264]
    buf = torch.full((rows, 288), 3.0, dtype=torch.bfloat16, device=dev)
    ops.linear(x, w, out=buf[:, 16:])
    assert torch.equal(buf[:, 16:], ops.linear(x.contiguous(), w))
    assert bool((buf[:, :16] == 3).all())
    dx = torch.full((rows, 272), 4.0, dtype=torch.bfloat16, device=dev)
    ops.linear_grad(buf[:, 16:], w, out=dx[:, 8:264])
    assert torch.equal(dx[:, 8:264], ops.linear_grad(buf[:, 16:].contiguous(), w))
    assert bool((dx[:, :8] == 4).all()) and bool((dx[:, 264:] == 4).all())


@pytest.mark.parametrize("call", ["linear", "linear_grad"])
@pytest.mark.parametrize("rows", [6, 150])
def test_bad_values_stay_in_their_rows(dev, rows, call):
    w = weights(dev, 1, 256, 256)
    ops = m.ExpertOps(1, 1, rows, 256)
    call = getattr(ops, call)
    x = torch.randn((rows, 256), generator=gen(dev, 1), device=dev).bfloat16()
    clean = call(x, w)
    x[1, 3], x[4, 255] = float("inf"), float("nan")
    y = call(x, w)
    assert bool(y[1].isnan().all()) and bool(y[4].isnan().all())
    keep = [r for r in range(rows) if r not in (1, 4)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("call", ["linear", "linear_grad"])
@pytest.mark.parametrize("rows", [3, 40, 500])
def test_repeats_bit_for_bit(dev, rows, call):
    w = weights(dev, 3, 1040, 1040)
    ops = m.ExpertOps(3, 1, rows, 1040)
    call = getattr(ops, call)
    x = torch.randn((rows, 1040), generator=gen(dev, 1), device=dev).bfloat16()
    starts = starts_of([rows // 3, 1, rows - rows // 3 - 1], dev)
    first = call(x, w, starts=starts)
    for _ in range(5):
        assert torch.equal(first, call(x, w, starts=starts))


@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [-5, 10, 20, 60], [0, 10, 20, 1 << 30],
                                 [70, 80, 90, 100], [60, 40, 20, 0]])
@pytest.mark.parametrize("call", ["linear", "linear_grad"])
def test_bad_starts_are_reported(dev, bad, call):
    w = weights(dev, 3, 128, 128)
    ops = m.ExpertOps(3, 1, 60, 128)
    x = torch.randn((60, 128), generator=gen(dev, 1), device=dev).bfloat16()
    buf = torch.full((62, 128), 3.0, dtype=torch.bfloat16, device=dev)
    getattr(ops, call)(x, w, starts=torch.tensor(bad, dtype=torch.int32, device=dev),
                       out=buf[1:61])
    assert ops.device_status() == m.MOE_ERR_INVALID_ARG
    assert ops.device_status() == m.MOE_OK
    assert bool((buf[0] == 3).all()) and bool((buf[61] == 3).all())
    y = ops.linear(x, w, starts=torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=dev))
    assert bool(torch.isfinite(y).all()) and ops.device_status() == m.MOE_OK


def test_starts_that_overlap_again_and_again(dev):
    """256 groups, every second of all rows: bounds that any sum of tiles would pass."""
    rows = 65536
    w = weights(dev, 256, 16, 16)
    ops = m.ExpertOps(256, 1, rows, 16)
    starts = torch.zeros(257, dtype=torch.int32, device=dev)
    starts[1::2] = rows
    x = torch.randn((rows, 16), generator=gen(dev, 1), device=dev).bfloat16()
    for call in (ops.linear, ops.linear_grad):
        buf = torch.full((rows + 2, 16), 3.0, dtype=torch.bfloat16, device=dev)
        call(x, w, starts=starts, out=buf[1:-1])
        assert ops.device_status() == m.MOE_ERR_INVALID_ARG
        assert bool((buf[0] == 3).all()) and bool((buf[-1] == 3).all())


def test_long_offsets(dev):
    """Rows and weights whose offsets pass 2^31."""
    rows, inner, out = 1 << 19, 4112, 48
    ops = m.ExpertOps(1, 8, 65536, 0)
    w = weights(dev, 1, out, inner)
    codes = torch.zeros((rows, inner), dtype=torch.uint8, device=dev)
    scales = torch.ones((rows, 33), device=dev)
    at = [0, 123456, 522199, 522200, rows - 1]
    codes[at] = torch.randint(0, 120, (5, inner), generator=gen(dev, 1), device=dev,
                              dtype=torch.int32).to(torch.uint8)
    y = ops.linear(m.QuantRows(codes, scales), w)
    few = ops.linear(m.QuantRows(codes[at].contiguous(), scales[at].contiguous()), w)
    # (other row counts may add the blocks in another order)
    assert bool((y[at].double() - few.double()).abs().max() <= 2 * R.BF16 * few.double().abs().max())
    y[at] = 0
    assert bool((y == 0).all())
    groups = 130                                 # weights of 2.1 GB, the last group's
    w = m.BlockWeights(torch.zeros((groups, 4096, 4096), dtype=torch.uint8, device=dev),
                       torch.ones((groups, 32, 32), device=dev))
    w.codes[groups - 1] = 0x38                   # 1.0
    x = torch.ones((2, 4096), dtype=torch.bfloat16, device=dev)
    starts = torch.zeros(groups + 1, dtype=torch.int32, device=dev)
    starts[groups] = 2
    ops = m.ExpertOps(groups, 1, 2, 4096)
    for call in (ops.linear, ops.linear_grad):
        y = call(x, w, starts=starts).double()
        # 448 codes of 1 / 448 each: the fp32 scale is within 2^-24 of 1 / 448
        assert bool(((y - 4096).abs() <= 4096 * R.BF16).all())
