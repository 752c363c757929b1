"""Row tiles at the number from which the prompt kernel takes over (needs a GB300)."""
from __future__ import annotations

import pytest

from test_gpu_attn import Case, dev, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,tiles", [(64, 2), (64, 3), (128, 3), (128, 4), (256, 5), (256, 6)])
@pytest.mark.parametrize("window", [0, 130])
def test_attention_at_the_kernels_border(dev, D, tiles, window):  # noqa: F811
    """Tiles of 16 rows (three tokens of five heads): the most that the decode kernel takes
    and the fewest of the prompt kernel, with one sequence, with two, and with keys shared
    out."""
    shape = m.AttnShape(q_heads=5, kv_heads=1, head_dim=D, page_tokens=32, rotary_dim=0,
                        window=window)
    for tokens in (3 * tiles, 3 * tiles + 1, 1000, 5000):
        Case(dev, shape, [(3 * tiles, tokens)], seed=tiles + tokens).check()
    if tiles % 2 == 0:
        Case(dev, shape, [(3 * tiles // 2, 700), (3 * tiles // 2, 90)], seed=tiles).check()
