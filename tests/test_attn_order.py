"""What the attention kernels' TMA warps publish, read from their source: a race between a
warp's lanes cannot be made to show itself, so its absence is checked where it would stand."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir,
                    "block_fp8_mixture_router_gb300", "csrc")


def body(file: str, function: str) -> str:
    """The text of a function's definition, comments taken out."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", re.search(rf"\b{function}\(const AttnArgs& a", text).end())
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i]


@pytest.mark.parametrize("file,function", [("k_attn_decode.cu", "produce"),
                                           ("k_attn_prompt.cu", "copy_tiles")])
def test_lanes_stores_are_ordered_before_one_lane_s_arrival(file, function):
    """Several lanes store a tile's scales and lane 0 alone arrives on the barrier that
    releases them: the others' stores are only covered with a __syncwarp() between (votes and
    reductions order no memory)."""
    text = body(file, function)
    last = [m.start() for m in re.finditer(r"sm\.meta\[[^;]*?=[^=]", text)]
    assert last
    arrive = text.index("mbar_arrive", last[-1])
    assert "__syncwarp()" in text[last[-1]:arrive]
