"""Inputs and outputs of the attention operators as column ranges of one buffer, which share
no byte (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_attn import Case, dev, m  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPE = m.AttnShape(q_heads=4, kv_heads=2, head_dim=64, page_tokens=16, rotary_dim=64)


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("rows,tokens", [(1, 40), (3, 90), (150, 170)])
def test_outputs_beside_the_inputs(dev, rows, tokens):  # noqa: F811
    """The same bits as with an output of its own, and nothing else of the buffer changes."""
    c = Case(dev, SHAPE, [(rows, tokens)], seed=rows)
    pos = torch.arange(tokens - rows, tokens, dtype=torch.int32, device=dev)
    packed = c.randn(rows, 4 + 2 + 2, 64)
    for name in ("forward", "rope", "step"):
        heads = 8 if name == "step" else 4
        buf = c.randn(rows, heads + 5, 64)               # the output, a head, the input
        x = buf[:, 5:5 + heads]
        x.copy_(packed[:, :heads])
        was = buf.clone()

        def call(x, out=None):
            if name == "forward":
                return c.net.forward(x, c.cache, c.batch, out=out)
            if name == "rope":
                return c.net.rope(x, pos, out=out)
            return c.net.step(x, c.cache, c.batch, out=out)
        if name == "step":
            call(x.contiguous())                         # (scales of the page have grown)
        want = call(x.contiguous())
        call(x, out=buf[:, :4])
        assert torch.equal(bits(buf[:, :4]), bits(want)), name
        assert torch.equal(bits(buf[:, 4:]), bits(was[:, 4:])), name
    assert c.net.device_status() == m.MOE_OK


def test_shared_bytes_are_refused(dev):  # noqa: F811
    c = Case(dev, SHAPE, [(3, 90)], seed=1)
    buf = c.randn(3, 12, 64)
    with pytest.raises(m.MoEError):
        c.net.forward(buf[:, 3:7], c.cache, c.batch, out=buf[:, :4])
    with pytest.raises(m.MoEError):
        c.net.forward(buf[:, :4], c.cache, c.batch, out=buf[:, 3:7])
    with pytest.raises(m.MoEError):
        c.net.step(buf[:, 3:11], c.cache, c.batch, out=buf[:, :4])
    pos = torch.arange(3, dtype=torch.int32, device=dev)
    with pytest.raises(m.MoEError):
        c.net.rope(buf[:, 1:5], pos, out=buf[:, :4])
    flat = buf.view(-1, 64)                              # rows of four and of six heads
    a = flat[:12].view(3, 4, 64)
    b = flat[6:24].view(3, 6, 64)[:, :4]
    with pytest.raises(m.MoEError):
        c.net.forward(a, c.cache, c.batch, out=b)
