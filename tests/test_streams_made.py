"""What the layer's, the chain's and the attention's calls return, and the copies they make of
rows that are not contiguous, are made under the stream the call was given, without a GPU."""
from __future__ import annotations

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe
from test_attn_devices import Library, ROWS, SHAPE, Stand, batch, cache, net  # noqa: F401
from test_ops_streams import GIVEN, OWN, Made, made  # noqa: F401


class Strided(Stand):
    """Rows with a gap behind each: a contiguous copy is a new tensor."""

    def is_contiguous(self):
        return False

    def contiguous(self):
        return torch.empty(tuple(self.shape), dtype=self.dtype, device=self.device)


@pytest.fixture
def layer(monkeypatch):
    lib = Library()
    monkeypatch.setattr(moe, "load_library", lambda: lib)
    monkeypatch.setattr(moe, "_ptr", lambda t: None)
    n = moe.MoELayer.__new__(moe.MoELayer)
    n.shape, n.max_rows, n.device, n.ctx = moe.LayerShape(hidden=256, top_k=4), 8, 0, None
    return n


def bf16(*shape, kind=Stand):
    return kind(torch.bfloat16, shape)


def layer_calls(layer, stream):
    x, g, rows = bf16(5, 256), bf16(256), bf16(5, 256, kind=Strided)
    kw = dict(stream=stream)
    chain = moe.MoEChain.__new__(moe.MoEChain)
    chain.layers, chain.chain = [layer, layer], None
    return {
        "forward": (1, lambda: layer.forward(x, **kw)),
        "forward of a copy": (2, lambda: layer.forward(rows, **kw)),
        "forward_addnorm": (3, lambda: layer.forward_addnorm(x, x, g, 1e-6, keep_xn=True, **kw)),
        "route": (3, lambda: layer.route(rows, **kw)),
        "quantize": (3, lambda: layer.quantize(rows, **kw)),
        "add_rmsnorm_quantize": (4, lambda: layer.add_rmsnorm_quantize(x, x, g, 1e-6, **kw)),
        "expert_activations": (2, lambda: layer.expert_activations(5, **kw)),
        "forward_codes": (2, lambda: layer.forward_codes(5, **kw)),
        "load": (8, lambda: layer.load({n: bf16(4, 4, kind=Strided) for n in (
            "w13", "s13", "w2", "s2", "router", "ws13", "ws2", "shared_gate")}, **kw)),
        "chain": (2, lambda: chain.forward(rows, **kw)),
    }


def attention_calls(net, stream):  # noqa: F811
    s, kw = SHAPE, dict(stream=stream)

    def rows(heads):
        return Stand(torch.bfloat16, (ROWS, heads, s.head_dim))
    return {
        "rope": (1, lambda: net.rope(rows(4), Stand(torch.int32, (ROWS,)), **kw)),
        "forward": (1, lambda: net.forward(rows(s.q_heads), cache(), batch(), **kw)),
        "step": (1, lambda: net.step(rows(s.q_heads + 2 * s.kv_heads), cache(), batch(), **kw)),
    }


@pytest.mark.parametrize("given, on, recorded", [
    (None, OWN, []), (OWN, OWN, []), (GIVEN, GIVEN, [OWN]), (0, 0, [OWN])])
def test_results_belong_to_the_stream(layer, net, made, given, on, recorded):  # noqa: F811
    for name, (count, call) in {**layer_calls(layer, given),
                                **attention_calls(net, given)}.items():
        made.clear()
        call()
        assert len(made) == count, name
        for t in made:
            assert t.on == on and t.recorded == recorded, name


def test_host_weights_stay_on_the_host(layer):
    """Copies of host tensors have no stream."""
    names = ("w13", "s13", "w2", "s2", "router", "ws13", "ws2", "shared_gate")
    layer.load({n: torch.zeros(4, 6).t() for n in names}, stream=GIVEN)
    assert all(t.is_contiguous() and not t.is_cuda for t in layer._keep)
