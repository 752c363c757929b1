"""The gated activation and its gradient where the sigmoid leaves fp32's normal range, against
the plain 64-bit form (tests/ops_reference.py) (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

import ops_reference as R
from test_gpu_ops_swiglu import sigmoid_bound

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")

LAST = 104.0           # e^-104 is below half of fp32's smallest subnormal
FAR = [-3e38, -1e36, -1e33, -1e6, -1000, -110, -LAST, -100, -95, -90, -89, -88.5, -88, -87.5, -87,
       -86, -81, -80, -79, -50, 50, 80, 87, 88, 89, 100, 110, 1000, 1e6, 1e33, 1e36, 3e38]
UPS = [1.0, -1.0, 1e-3, 1e30, -3e38, 0.0]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


def lost(g):
    """What the smaller of sigmoid(z) and sigmoid(-z) loses below fp32's normal range, and its
    product with the gate: e^-|z| a subnormal step, its product with 1 / (1 + e^-|z|) half of
    one, times the gate, and half a step of that product.  Behind the last subnormal it is 0, and
    0 times the gate."""
    return 2.0 ** -148 * (g.abs().clamp(max=LAST) + 1)


def slack(g):
    return sigmoid_bound(g.clamp(-LAST, LAST))   # (behind it e^-|z| is 0 and nothing is lost)


def gates(dev, up, big=False):
    """One row: every far gate that has a finite result (or is large on purpose) with this up."""
    g = torch.tensor([v for v in FAR if big or v < 1e3 or abs(up) <= 1], dtype=torch.float32,
                     device=dev)
    g = torch.nn.functional.pad(g, (0, -g.numel() % 16))
    return torch.cat([g, torch.full_like(g, up)])[None].bfloat16()


@pytest.mark.parametrize("up", UPS)
def test_forward(dev, up):
    gu = gates(dev, up)
    g, u = gu.double().chunk(2, dim=1)
    want = R.swiglu(gu)
    fits = want.abs() < 2.0 ** 127
    y = m.ExpertOps(1, 1, 1, 0).swiglu(gu).double()
    allowed = (R.BF16 * (1 + 2.0 ** -7) + slack(g)) * want.abs() + lost(g) * u.abs() + 2.0 ** -134
    assert bool(((y - want).abs() <= allowed)[fits].all())
    assert bool((y[g < -LAST] == 0).all())


@pytest.mark.parametrize("up", UPS)
@pytest.mark.parametrize("d", [1.0, -1e-3])
def test_gradient(dev, up, d):
    gu = gates(dev, up)
    g, u = gu.double().chunk(2, dim=1)
    dh = torch.full(g.shape, d, dtype=torch.bfloat16, device=dev)
    want, dd = R.swiglu_grad(dh, gu), dh.double()
    fits = want.abs() < 2.0 ** 127
    s = torch.sigmoid(g)
    got = m.ExpertOps(1, 1, 1, 0).swiglu_grad(dh, gu).double()
    # dgate's two terms, s and g s sigmoid(-g), may cancel: relative to their magnitudes
    terms = torch.cat([dd.abs() * u.abs() * (s + (g * s).abs() * torch.sigmoid(-g)),
                       want[:, g.shape[1]:].abs()], 1)
    rel, gone = torch.cat([slack(g)] * 2, 1), torch.cat([lost(g)] * 2, 1)
    size = torch.cat([dd.abs() * u.abs(), dd.abs()], 1)
    allowed = (R.BF16 * (1 + 2.0 ** -7) * want.abs() + 2 * rel * terms + 2 * gone * size +
               2.0 ** -134)
    assert bool(((got - want).abs() <= allowed)[fits].all())
    below = torch.cat([g < -LAST] * 2, 1)
    assert bool((got[below] == 0).all())


@pytest.mark.parametrize("gate", [-3e38, -1e33, -200.0])
def test_neighbours_in_codes(dev, gate):
    """A far gate sets no scale: its group's codes are those of a zero in its place."""
    gen = torch.Generator(dev).manual_seed(3)
    gu = torch.randn((2, 512), generator=gen, device=dev).bfloat16()
    dh = torch.randn((2, 256), generator=gen, device=dev).bfloat16()
    ops = m.ExpertOps(1, 1, 2, 0)
    far, none = gu.clone(), gu.clone()
    far[1, 130], none[1, 130] = gate, 0.0
    a, b = ops.swiglu(far, quantize=True), ops.swiglu(none, quantize=True)
    assert torch.equal(a.scales, b.scales)
    assert torch.equal(a.codes & 127, b.codes & 127)         # (a zero's sign is the up's)
    down = dh.clone()
    down[1, 130] = 0.0
    a, b = ops.swiglu_grad(dh, far, quantize=True), ops.swiglu_grad(down, none, quantize=True)
    assert torch.equal(a.scales, b.scales) and torch.equal(a.codes & 127, b.codes & 127)


def test_infinite_and_no_numbers(dev):
    inf, nan = float("inf"), float("nan")
    gu = torch.tensor([[-inf, inf, nan] + [1.0] * 13 + [1.0] * 16], device=dev).bfloat16()
    ops = m.ExpertOps(1, 1, 1, 0)
    y = ops.swiglu(gu)[0]
    assert bool(y[[0, 2]].isnan().all()) and float(y[1]) == inf
    d = ops.swiglu_grad(torch.ones((1, 16), dtype=torch.bfloat16, device=dev), gu)[0]
    assert bool(d[[0, 1, 2, 16, 18]].isnan().all()) and float(d[17]) == inf
    assert bool(torch.isfinite(y[3:]).all()) and bool(torch.isfinite(d[3:16]).all())
