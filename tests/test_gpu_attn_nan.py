"""A value row with a NaN in some of its columns, as other code than the append may leave
one: every row that sees it is NaN throughout, wherever its token lies (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_attn import Case, check_close, dev, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw,rows,tokens", [
    (dict(q_heads=4, kv_heads=2, head_dim=128, page_tokens=64), 1, 700),
    (dict(q_heads=16, kv_heads=1, head_dim=64, page_tokens=16), 1, 500),
    (dict(q_heads=3, kv_heads=1, head_dim=256, page_tokens=32), 4, 600),
    (dict(q_heads=8, kv_heads=2, head_dim=128, page_tokens=64), 1, 9000),   # keys shared out
    (dict(q_heads=4, kv_heads=2, head_dim=64, page_tokens=32), 200, 600),
    (dict(q_heads=4, kv_heads=2, head_dim=128, page_tokens=128), 300, 900),
    (dict(q_heads=8, kv_heads=4, head_dim=256, page_tokens=64), 140, 700),
    (dict(q_heads=8, kv_heads=1, head_dim=128, page_tokens=64), 150, 6000)])
@pytest.mark.parametrize("token", [0, 200, -70, -2])
def test_one_nan_value_makes_its_rows_nan(dev, kw, rows, tokens, token):  # noqa: F811
    shape = m.AttnShape(rotary_dim=0, **kw)
    c = Case(dev, shape, [(rows, tokens)], seed=tokens)
    q = c.q()
    plain = c.check(q).clone()
    token %= tokens
    P, g = shape.page_tokens, shape.q_heads // shape.kv_heads
    head = shape.kv_heads - 1
    c.codes["v"][int(c.pages[0, token // P]), head, token % P, shape.head_dim - 3] = 0xFF
    out = c.net.forward(q, c.cache, c.batch)
    want = plain.clone()
    want[max(0, token - (tokens - rows)):, head * g:] = float("nan")
    check_close(out, want.double(), torch.zeros_like(want, dtype=torch.float64))
    assert c.net.device_status() == m.MOE_OK
