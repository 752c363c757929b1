"""Rows of no group, in front of the first start, behind the last and behind an order's last row,
may hold anything: nothing depends on them and they stay as they were (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

import ops_reference as R
from test_gpu_ops_linear import bound, gen, weights

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("starts, rows", [
    ([5, 12, 12, 40], 60), ([3, 4, 4, 4], 9), ([31, 200, 331, 331], 400), ([7, 7, 7, 7], 20)],
    ids=str)
def test_products(dev, starts, rows, trans, quantized):
    for out, inner in ((128, 256), (1552, 1808)):       # both kernels of the forward product
        w = weights(dev, 3, out, inner)
        K, N = (out, inner) if trans else (inner, out)
        x = torch.randn((rows, K), generator=gen(dev, 1), device=dev).bfloat16()
        codes, scales = R.quantise(x)
        bad = torch.ones(rows, dtype=torch.bool, device=dev)
        bad[starts[0]:starts[-1]] = False
        x[bad], codes[bad], scales[bad] = float("nan"), 0x7F, float("inf")
        ops = m.ExpertOps(3, 1, rows, 0 if quantized else K)
        y = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device=dev)
        at = torch.tensor(starts, dtype=torch.int32, device=dev)
        (ops.linear_grad if trans else ops.linear)(m.QuantRows(codes, scales) if quantized else x,
                                                   w, starts=at, out=y)
        want, mag = R.linear(R.values(codes, scales), w.codes, w.scales, starts,
                             torch.full_like(y, -77.0), trans)
        err = (y.double() - want).abs()
        assert bool((err <= bound(K) * mag + R.BF16 * (1 + 2.0 ** -7) * want.abs()).all())
        assert bool((y[bad] == -77).all())
        assert ops.device_status() == m.MOE_OK


@pytest.mark.parametrize("tokens", [6, 2000])
def test_back_to_tokens(dev, tokens):
    k, E, H = 8, 16, 264
    ops = m.ExpertOps(E, k, tokens, 0)
    idx = torch.randint(-8, E, (tokens, k), generator=gen(dev, 2), device=dev, dtype=torch.int32)
    order = ops.sort(idx)
    kept = int(order.starts[-1])
    rows = torch.randn((tokens * k, H), generator=gen(dev, 3), device=dev).bfloat16()
    dy = torch.randn((tokens, H), generator=gen(dev, 4), device=dev).bfloat16()
    w = torch.rand((tokens, k), generator=gen(dev, 5), device=dev)

    def all_of(r):
        out = torch.full((tokens * k, H), -77.0, dtype=torch.bfloat16, device=dev)
        drows, dw = ops.combine_grad(dy, r, order, w, out=out)
        return ops.dispatch_grad(r, order), ops.combine(r, order, w), drows, dw
    want = all_of(rows)
    rows[kept:] = float("nan")
    got = all_of(rows)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((got[2][kept:] == -77).all()) and ops.device_status() == m.MOE_OK
