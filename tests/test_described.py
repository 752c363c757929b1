"""Objects that describe tensors to the C calls hold their addresses: another tensor put into an
attribute would go unseen, and is refused (no GPU: stand-ins)."""
from __future__ import annotations

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe
from test_attn_devices import Stand, batch, cache
from test_ops_devices import E, H, K, N, T, quant


@pytest.mark.parametrize("what, names", [
    (lambda: quant(T, H), ("codes", "scales", "shape", "device")),
    (lambda: moe.BlockWeights(Stand(torch.uint8, (E, N, H)), Stand(torch.float32, (E, 1, 1))),
     ("codes", "scales", "groups", "out", "inner")),
    (lambda: moe.ExpertOrder(*[Stand3(n) for n in ((E + 1,), (T * K,), (T, K))]),
     ("starts", "pair_of_slot", "slot_of_pair", "tokens")),
    (cache, ("k_codes", "v_codes", "k_scales", "v_scales")),
    (batch, ("row_start", "kv_len", "pages", "rows"))],
    ids=["QuantRows", "BlockWeights", "ExpertOrder", "KVCache", "AttnBatch"])
def test_attributes_are_fixed(what, names):
    t = what()
    for n in names:
        was = getattr(t, n)
        with pytest.raises(AttributeError):
            setattr(t, n, was)
        assert getattr(t, n) is was


class Stand3(Stand):
    def __init__(self, shape):
        super().__init__(torch.int32, shape)

    def numel(self):
        return self.t.numel()
