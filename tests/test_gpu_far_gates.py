"""Experts whose gates lie far below zero add nothing to the layer's output, on every path
(needs a GB300)."""
from __future__ import annotations

import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


def far_layer(shape, part, dev):
    """A layer whose routed or shared gates are all near -1e33 for rows of positive values, and
    that layer with the part's down projection zero."""
    layer = W.make_layer(shape, 5, "bias_skew", device=dev)
    none = None
    if part == "routed":
        layer["w13"][:, :shape.inter] = 0xB8                       # -1.0
        layer["s13"][:, :shape.inter // shape.group] = 1e33 / shape.hidden
        none = dict(layer, w2=torch.zeros_like(layer["w2"]))
    else:
        layer["ws13"][:shape.shared_inter] = -1e33 / shape.hidden
        none = dict(layer, ws2=torch.zeros_like(layer["ws2"]))
    return layer, none


@pytest.mark.parametrize("part", ["routed", "shared"])
@pytest.mark.parametrize("shape", [W.TINY, W.FULL], ids=["tiny", "full"])
def test_far_gates_add_nothing(dev, shape, part):
    rows = (1, 2, 4, 8, 11, 16, 40, 300)
    nets = []
    for layer in far_layer(shape, part, dev):
        nets.append(m.MoELayer(m.LayerShape(shape.hidden, shape.n_experts, shape.top_k,
                                            shape.inter, shape.shared_inter), max(rows)))
        nets[-1].load(layer)
    for T in rows:
        x = W.make_x(shape, T, 7, "bias_skew", device=dev).abs() + 0.125
        y, want = nets[0].forward(x), nets[1].forward(x)
        assert bool(torch.isfinite(want).all()) and bool((want != 0).any())
        assert torch.equal(y, want), (T, float((y.double() - want.double()).abs().max()))
        assert nets[0].device_status() == m.MOE_OK
    for n in nets:
        n.close()
