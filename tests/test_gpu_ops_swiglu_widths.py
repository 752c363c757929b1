"""The gated activation's gradient to codes where a lane's sixteen columns hold gates and ups: widths
that are multiples of 8 but not of 16 (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

import ops_reference as R
from test_gpu_ops_swiglu import inputs, sigmoid_bound

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


@pytest.mark.parametrize("size", [(1, 8), (5, 24), (33, 56), (2, 72), (7, 120), (9, 136), (300, 1000),
                                  (3, 1016), (3, 1040), (2, 65528)], ids=str)
def test_against_the_formula(dev, size):
    rows, width = size
    gu, dh = inputs(dev, rows, width)
    g, u = gu.double().chunk(2, dim=1)
    want, s = R.swiglu_grad(dh, gu), torch.sigmoid(g)
    rel = torch.cat([sigmoid_bound(g)] * 2, 1)
    mag = torch.cat([dh.double().abs() * u.abs() * (s + (g * s).abs()), want[:, width:].abs()], 1)
    codes = torch.full((rows + 1, 2 * width), 0x55, dtype=torch.uint8, device=dev)
    scales = torch.full((rows + 1, -(-2 * width // 128)), 9.0, device=dev)
    ops = m.ExpertOps(1, 1, rows, 0)
    got = ops.swiglu_grad(dh, gu, out=m.QuantRows(codes[:rows], scales[:rows]))
    assert bool((codes[rows] == 0x55).all()) and bool((scales[rows] == 9).all())
    v = R.values(got.codes, got.scales)
    sc = got.scales.double().repeat_interleave(128, dim=1)[:, :2 * width]
    # half a step of the code, of a value known to rel of its terms; the scale's own quotient
    # and the values' are rounded to fp32
    half = torch.maximum(R.E4M3 * want.abs(), R.E4M3_SUB * sc)
    assert bool(((v - want).abs() <= half * (1 + 2.0 ** -4) + 4 * rel * mag).all())
    amax = torch.nn.functional.pad(want.abs(), (0, -2 * width % 128)).view(rows, -1, 128).amax(2)
    off = torch.nn.functional.pad(2 * rel * mag, (0, -2 * width % 128)).view(rows, -1, 128).amax(2)
    assert bool(((got.scales.double() * 448 - amax).abs() <= off + 2.0 ** -22 * amax).all())
    assert ops.device_status() == m.MOE_OK


def test_strides_and_other_widths(dev):
    """Columns of wider buffers; h itself in codes still wants whole vectors of 16."""
    gu, dh = inputs(dev, 20, 64)
    ops = m.ExpertOps(1, 1, 20, 0)
    a = ops.swiglu_grad(dh[:, 8:48], gu[:, 16:96], quantize=True)
    b = ops.swiglu_grad(dh[:, 8:48].contiguous(), gu[:, 16:96].contiguous(), quantize=True)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    for call in (lambda: ops.swiglu(gu[:, :80], quantize=True),
                 lambda: ops.swiglu_grad(dh[:, :36], gu[:, :72], quantize=True)):
        with pytest.raises(m.MoEError) as e:
            call()
        assert e.value.status == m.MOE_ERR_INVALID_ARG
