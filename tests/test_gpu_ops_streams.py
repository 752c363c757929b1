"""Results of calls on a stream given by hand, beside a caller's stream that is busy with memory
freed a moment ago (needs a GB300)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")

BUSY = 100_000_000       # clocks: some 50 ms


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


@pytest.fixture(params=["stream", "handle"])
def side(request, dev):
    s = torch.cuda.Stream()
    yield s, (s if request.param == "stream" else s.cuda_stream)
    torch.cuda.synchronize()


def test_not_of_memory_that_the_caller_still_writes(dev, side):
    s, given = side
    ops = m.ExpertOps(1, 1, 512, 0)
    gu = torch.randn((512, 2048), device=dev).bfloat16()
    want = ops.swiglu(gu)
    torch.cuda.synchronize()
    old = torch.empty_like(want)
    at = old.data_ptr()
    torch.cuda._sleep(BUSY)
    old.fill_(7.0)
    del old
    got = ops.swiglu(gu, stream=given)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_held_until_the_caller_has_read_it(dev, side):
    s, given = side
    ops = m.ExpertOps(1, 1, 512, 0)
    gu = torch.randn((512, 2048), device=dev).bfloat16()
    want = ops.swiglu(gu)
    torch.cuda.synchronize()
    got = ops.swiglu(gu, stream=given)
    s.synchronize()
    torch.cuda._sleep(BUSY)
    copy = got.clone()
    del got
    with torch.cuda.stream(s if not isinstance(given, int) else
                           torch.cuda.ExternalStream(given)):
        torch.empty_like(want).fill_(7.0)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_the_parts_on_a_stream_given_by_hand(dev, side):
    """Every result of a forward and a backward made on that stream."""
    s, given = side
    T, k, E, H, I = 40, 4, 16, 256, 128
    ops = m.ExpertOps(E, k, T, H)
    g = torch.Generator(dev).manual_seed(0)
    w13, w2 = (m.BlockWeights(torch.randint(0, 120, (E, o, i), generator=g, device=dev,
                                            dtype=torch.int32).to(torch.uint8),
                              torch.full((E, o // 128, i // 128), 1e-3, device=dev))
               for o, i in ((2 * I, H), (H, I)))
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    dy = torch.randn((T, H), generator=g, device=dev).bfloat16()
    idx = torch.randint(0, E, (T, k), generator=g, device=dev, dtype=torch.int32)
    w = torch.rand((T, k), generator=g, device=dev)

    def both(on):
        order, rows = ops.dispatch(x, idx, stream=on)
        st = order.starts
        gu = ops.linear(rows, w13, starts=st, stream=on)
        out = ops.linear(ops.swiglu(gu, quantize=True, stream=on), w2, starts=st, stream=on)
        y = ops.combine(out, order, w, stream=on)
        dout, dw = ops.combine_grad(dy, out, order, w, quantize=True, stream=on)
        dgu = ops.swiglu_grad(ops.linear_grad(dout, w2, starts=st, stream=on), gu, stream=on)
        return y, dw, ops.dispatch_grad(ops.linear_grad(dgu, w13, starts=st, stream=on), order,
                                        stream=on)
    want = both(None)
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(BUSY)
    got = both(given)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ops.device_status() == m.MOE_OK


def test_a_branch_of_a_captured_graph(dev, side):
    """A stream given by hand that the capture has forked to: replayed with other rows."""
    s, given = side
    ops = m.ExpertOps(1, 1, 512, 0)
    gu = torch.randn((512, 2048), device=dev).bfloat16()
    dh = torch.randn((512, 1024), device=dev).bfloat16()
    ops.swiglu(gu, stream=given)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        y = ops.swiglu(gu, stream=given)
        d = ops.swiglu_grad(dh, gu, quantize=True, stream=given)
        torch.cuda.current_stream().wait_stream(s)
        z = y + 1
    for seed in range(3):
        torch.manual_seed(seed)
        gu.copy_(torch.randn(gu.shape, device=dev))
        graph.replay()
        want, dwant = ops.swiglu(gu), ops.swiglu_grad(dh, gu, quantize=True)
        assert torch.equal(y, want) and torch.equal(z, want + 1)
        assert torch.equal(d.codes, dwant.codes) and torch.equal(d.scales, dwant.scales)
