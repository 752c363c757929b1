"""The attention operators beside the MoE layer, as examples/backbone_blocks.py runs them
(needs a GB300)."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import attn_reference as R
import workloads as W

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")

sys.path.insert(0, os.path.join(os.path.dirname(__file__), os.pardir, "examples"))

import backbone_blocks as B  # noqa: E402

SHAPE = m.AttnShape(q_heads=8, kv_heads=2, head_dim=64, page_tokens=16, rotary_dim=32)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


def test_block_is_its_parts(dev):
    """Prompts of 40 and 7 rows, then a row each: a block's output is, bit for bit, the
    add-norm, the projections, the attention step and the MoE layer one after the other,
    and the step's attention is the plain form's over the cache that it left."""
    net = B.Backbone(SHAPE, W.TINY, blocks=1, seqs=2, most_tokens=64, max_rows=47, device=dev)
    block, pages = net.blocks[0], net.pages
    twin = m.KVCache.empty(SHAPE, pages.n_pages, dev)
    for rows, seed in (([40, 7], 1), ([1, 1], 2)):
        n = sum(rows)
        pages.kv_len += torch.tensor(rows, dtype=torch.int32, device=dev)
        batch = pages.batch(rows)
        r, x, _ = (t.to(dev) for t in W.make_addnorm(W.TINY, n, seed))
        h, y = block.forward(r, x, batch)

        h1, xn, _, _ = block.moe.add_rmsnorm_quantize(r, x, block.norm_in, B.EPS)
        qkv = (xn @ block.w_qkv).view(n, -1, SHAPE.head_dim)
        pos = torch.cat([torch.arange(k - i, k) for i, k in zip(rows, pages.kv_len.tolist())])
        pos = pos.to(torch.int32).to(dev)
        hq, hk = SHAPE.q_heads, SHAPE.kv_heads
        q = net.attn.rope(qkv[:, :hq], pos, gamma=block.norm_q, eps=B.EPS)
        k = net.attn.rope(qkv[:, hq:hq + hk], pos, gamma=block.norm_k, eps=B.EPS)
        net.attn.append(k, qkv[:, hq + hk:], twin, batch)
        out = net.attn.forward(q, twin, batch)
        h2, _, y2 = block.moe.forward_addnorm(h1, out.view(n, -1) @ block.w_out,
                                              block.norm_moe, B.EPS)
        assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
        assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
        want, tol = R.attention(SHAPE, q, block.cache.k_codes, block.cache.k_scales,
                                block.cache.v_codes, block.cache.v_scales, pages.table,
                                batch.row_start, pages.kv_len)
        assert bool(((out.double() - want).abs() <= tol).all())
    net.check()


def test_example_runs(dev, capsys):
    B.main(steps=4)
    assert "us a block" in capsys.readouterr().out
