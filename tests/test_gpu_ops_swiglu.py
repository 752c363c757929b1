"""The gated activation and its gradient on the GPU against the plain 64-bit form
(tests/ops_reference.py) (needs a GB300)."""
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


def inputs(dev, rows, width, spread=3.0):
    g = torch.Generator(device=dev)
    g.manual_seed(rows + width)
    gu = spread * torch.randn((rows, 2 * width), generator=g, device=dev)
    return gu.bfloat16(), torch.randn((rows, width), generator=g, device=dev).bfloat16()


def sigmoid_bound(z):
    """e^-z by the fast exponential (2 + 1.173 |z| ulps of 2^-23), 1 + it, a quotient (2 ulps)
    and the products around it: relative to silu."""
    return (12 + 1.2 * z.abs()) * 2.0 ** -23


def close_codes(got, want, rel):
    """Codes x scales within half a step of the values, which are known to `rel`."""
    v = R.values(got.codes, got.scales)
    s = got.scales.double().repeat_interleave(128, dim=1)[:, :want.shape[1]]
    slack = rel + 2.0 ** -22
    half = torch.maximum(R.E4M3 * want.abs(), R.E4M3_SUB * s)
    assert bool(((v - want).abs() <= half * (1 + 2.0 ** -4) + slack * want.abs()).all())
    amax = torch.nn.functional.pad(want.abs(), (0, -want.shape[1] % 128)).view(
        want.shape[0], -1, 128).amax(2)
    there = amax > 0
    err = (got.scales.double() - amax / 448).abs() / (amax / 448).clamp(min=1e-300)
    assert bool((err[there] <= float(rel.max()) + 2.0 ** -22).all())


SIZES = [(1, 512), (1, 16), (3, 128), (17, 1408), (200, 272), (1000, 512), (5, 4096)]


@pytest.mark.parametrize("size", SIZES + [(9, 8), (31, 1000)], ids=str)
def test_swiglu(dev, size):
    gu, dh = inputs(dev, *size)
    ops = m.ExpertOps(1, 1, size[0], 0)
    z = gu[:, :size[1]].double()
    want, rel = R.swiglu(gu), sigmoid_bound(z)
    err = (ops.swiglu(gu).double() - want).abs()
    assert bool((err <= (R.BF16 * (1 + 2.0 ** -7) + rel) * want.abs()).all())
    if size[1] % 16 == 0:
        close_codes(ops.swiglu(gu, quantize=True), want, rel)


@pytest.mark.parametrize("size", SIZES + [(9, 8), (31, 1000)], ids=str)
def test_swiglu_grad(dev, size):
    gu, dh = inputs(dev, *size)
    ops = m.ExpertOps(1, 1, size[0], 0)
    g, u = gu.double().chunk(2, dim=1)
    want, s = R.swiglu_grad(dh, gu), torch.sigmoid(g)
    rel = sigmoid_bound(g)
    # dgate = dh u (s + z (1 - s)): the two terms may cancel, so relative to their sum
    mag = torch.cat([dh.double().abs() * u.abs() * (s + (g * s).abs()), want[:, size[1]:].abs()], 1)
    rel = torch.cat([rel, rel], 1)
    err = (ops.swiglu_grad(dh, gu).double() - want).abs()
    assert bool((err <= R.BF16 * (1 + 2.0 ** -7) * want.abs() + 2 * rel * mag).all())
    if size[1] % 16 == 0:
        got = ops.swiglu_grad(dh, gu, quantize=True)
        v = R.values(got.codes, got.scales)
        sc = got.scales.double().repeat_interleave(128, dim=1)[:, :2 * size[1]]
        half = torch.maximum(R.E4M3 * want.abs(), R.E4M3_SUB * sc)
        assert bool(((v - want).abs() <= half * (1 + 2.0 ** -4) + 4 * rel * mag).all())


def test_gradient_is_the_derivative():
    """The formula against autograd and against differences, in 64 bits."""
    torch.manual_seed(0)
    gu = (3 * torch.randn(4, 10, dtype=torch.float64)).requires_grad_()
    dh = torch.randn(4, 5, dtype=torch.float64)
    got = R.swiglu_grad(dh, gu.detach())
    auto, = torch.autograd.grad((R.swiglu(gu) * dh).sum(), gu)
    assert torch.allclose(got, auto, rtol=1e-12, atol=1e-12)
    for i in range(4):
        for c in range(10):
            e = torch.zeros(4, 10, dtype=torch.float64)
            e[i, c] = 1e-6
            d = ((R.swiglu(gu + e) - R.swiglu(gu - e)) * dh).sum() / 2e-6
            assert abs(float(d - got[i, c])) < 1e-7


def test_far_gates(dev):
    """Gates to both ends: the sigmoid is 0 or 1, nothing overflows."""
    g = torch.tensor([-3e38, -1000, -89, -88, -20, -1, -0.0, 0.0, 1, 20, 89, 1000, 3e38],
                     device=dev)
    gu = torch.cat([g.repeat(1, 1), torch.ones((1, 13), device=dev)], 1)
    gu = torch.cat([torch.nn.functional.pad(gu[:, :13], (0, 3)),
                    torch.nn.functional.pad(gu[:, 13:], (0, 3))], 1).bfloat16()
    ops = m.ExpertOps(1, 1, 1, 0)
    y = ops.swiglu(gu)[0].double()
    want = R.swiglu(gu)[0]
    # below -80 the sigmoid is held at e^-80, 1.8e-35
    assert bool(((y - want).abs() <= 2 * R.BF16 * want.abs() + 2e-35 * gu[0, :16].double().abs()
                 ).all())
    d = ops.swiglu_grad(torch.ones((1, 16), dtype=torch.bfloat16, device=dev), gu)
    assert bool(torch.isfinite(d).all()) and float(d[0, 11]) == 1.0 and abs(float(d[0, 1])) < 1e-30


def test_strides_and_other_rows(dev):
    ops = m.ExpertOps(1, 1, 40, 0)
    wide, dh = inputs(dev, 40, 80)
    buf = torch.full((40, 136), 9.0, dtype=torch.bfloat16, device=dev)
    gu = wide[:, 32:32 + 96]
    ops.swiglu(gu, out=buf[:, 8:56])
    assert torch.equal(buf[:, 8:56], ops.swiglu(gu.contiguous()))
    ops.swiglu_grad(dh[:, 16:64], gu, out=buf[:, 40:136])
    assert torch.equal(buf[:, 40:136], ops.swiglu_grad(dh[:, 16:64].contiguous(), gu.contiguous()))
    assert bool((buf[:, :8] == 9).all())
