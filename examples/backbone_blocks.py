"""A backbone of a few blocks, served: two prompts in one batch, then one row for each of
them per step, replayed as a CUDA graph.

A block adds the block before it to the residual stream and norms it, projects to query,
key and value heads, takes the attention step (norm and rotary positions of the heads,
append to the 8-bit paged cache, attention), projects back, and hands residual and output
to the MoE layer with its own add-norm.  Weights are random; the projections are plain
matrix products.

    python examples/backbone_blocks.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_fp8_mixture_router_gb300 as moe  # noqa: E402
import workloads as W  # noqa: E402

EPS = W.NORM_EPS


class Pages:
    """Which pages hold which sequence's tokens, and how many tokens each has."""

    def __init__(self, seqs: int, most_tokens: int, page_tokens: int, device):
        per = -(-most_tokens // page_tokens)
        self.n_pages, self.seqs, self.most = seqs * per, seqs, most_tokens
        # (any order will do; a server hands pages out as sequences grow)
        order = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(0))
        self.table = order.to(torch.int32).view(seqs, per).to(device)
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device=device)

    def batch(self, rows: list[int]) -> moe.AttnBatch:
        """A call of rows[s] new tokens for sequence s; kv_len has to count them by the time
        it runs."""
        start = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32)
        return moe.AttnBatch(start.to(self.table.device), self.kv_len, self.table, sum(rows),
                             max_seq_rows=max(rows), max_kv_len=self.most)


class Block:
    def __init__(self, attn: moe.Attention, shape: W.MoEShape, pages: Pages, seed: int,
                 max_rows: int, device):
        s, H = attn.shape, shape.hidden
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*size, scale):
            return (scale * torch.randn(size, generator=g, device=device)).to(torch.bfloat16)
        self.attn = attn
        self.w_qkv = randn(H, (s.q_heads + 2 * s.kv_heads) * s.head_dim, scale=H ** -0.5)
        self.w_out = randn(s.q_heads * s.head_dim, H, scale=(s.q_heads * s.head_dim) ** -0.5)
        self.norm_in, self.norm_moe = 1 + randn(2, H, scale=0.1)
        self.norm_q, self.norm_k = 1 + randn(2, s.head_dim, scale=0.1)
        self.cache = moe.KVCache.empty(s, pages.n_pages, device)
        self.moe = moe.MoELayer(moe.LayerShape(shape.hidden, shape.n_experts, shape.top_k,
                                               shape.inter, shape.shared_inter), max_rows)
        self.moe.load(W.make_layer(shape, seed, device=device))

    def forward(self, h: torch.Tensor, x: torch.Tensor, batch: moe.AttnBatch):
        """Residual stream and the block before's output: the new ones."""
        h, xn, _, _ = self.moe.add_rmsnorm_quantize(h, x, self.norm_in, EPS)
        qkv = (xn @ self.w_qkv).view(batch.rows, -1, self.attn.shape.head_dim)
        out = self.attn.step(qkv, self.cache, batch, q_gamma=self.norm_q, k_gamma=self.norm_k,
                             eps=EPS)
        h, _, y = self.moe.forward_addnorm(h, out.view(batch.rows, -1) @ self.w_out,
                                           self.norm_moe, EPS)
        return h, y


class Backbone:
    def __init__(self, attn_shape: moe.AttnShape, shape: W.MoEShape, blocks: int, seqs: int,
                 most_tokens: int, max_rows: int, device="cuda"):
        self.pages = Pages(seqs, most_tokens, attn_shape.page_tokens, device)
        # one workspace for all blocks: they run one after the other
        self.attn = moe.Attention(attn_shape, max_rows=max_rows, max_seqs=seqs)
        self.blocks = [Block(self.attn, shape, self.pages, 100 + i, max_rows, device)
                       for i in range(blocks)]

    def forward(self, x: torch.Tensor, batch: moe.AttnBatch) -> torch.Tensor:
        h = torch.zeros_like(x)
        for b in self.blocks:
            h, x = b.forward(h, x, batch)
        return h + x

    def check(self):
        status = self.attn.device_status()
        if status != moe.MOE_OK:
            raise moe.MoEError(status, "attention")


def main(steps: int = 32):
    device = torch.device("cuda", 0)
    torch.cuda.set_device(device)
    attn_shape = moe.AttnShape(q_heads=16, kv_heads=2, head_dim=128, page_tokens=64,
                               rotary_dim=32)
    prompts = [300, 45]
    net = Backbone(attn_shape, W.FULL, blocks=2, seqs=2, most_tokens=300 + steps,
                   max_rows=sum(prompts), device=device)
    pages = net.pages

    pages.kv_len += torch.tensor(prompts, dtype=torch.int32, device=device)
    y = net.forward(W.make_x(W.FULL, sum(prompts), 1, device=device), pages.batch(prompts))
    net.check()
    rows = y[[prompts[0] - 1, sum(prompts) - 1]].clone()  # each prompt's last row goes on
    scale = rows.float().norm(dim=1, keepdim=True)

    one = pages.batch([1, 1])

    def step():
        pages.kv_len.add_(1)
        out = net.forward(rows, one).float()
        rows.copy_(out * (scale / out.norm(dim=1, keepdim=True)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    a.record()
    for _ in range(steps - 1):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    net.check()
    assert pages.kv_len.tolist() == [n + steps for n in prompts]
    assert bool(torch.isfinite(rows).all())
    print(f"{steps} rows for each of {len(prompts)} sequences, "
          f"{a.elapsed_time(b) / max(steps - 1, 1) * 1e3 / len(net.blocks):.1f} us a block")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 32)
