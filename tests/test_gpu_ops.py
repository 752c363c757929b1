"""The layer's parts together, as a program uses them: forward against the whole layer,
backward stage by stage, captured and replayed, on other streams; and their refusals (needs a
GB300)."""
from __future__ import annotations

import ctypes
import os
import sys

import pytest
import torch

import ops_reference as R
import workloads as W

pytestmark = pytest.mark.gpu

m = pytest.importorskip("block_fp8_mixture_router_gb300")

sys.path.insert(0, os.path.join(os.path.dirname(__file__), os.pardir, "examples"))

import expert_parts as P  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    return torch.device("cuda", 0)


def make(dev, shape, tokens, seed=0, quantize=True, kind="normal"):
    layer = W.make_layer(shape, seed, kind, device=dev)
    for n in ("ws13", "ws2"):
        layer[n].zero_()                        # no shared expert: the routed half alone
    net = m.MoELayer(m.LayerShape(shape.hidden, shape.n_experts, shape.top_k, shape.inter,
                                  shape.shared_inter), tokens)
    net.load(layer)
    return net, P.Experts(shape, layer, tokens, quantize)


@pytest.mark.parametrize("quantize", [True, False])
@pytest.mark.parametrize("tokens", [1, 3, 11, 300])
def test_forward_is_the_layer(dev, tokens, quantize):
    net, parts = make(dev, W.TINY, tokens, quantize=quantize)
    x = W.make_x(W.TINY, tokens, 1, device=dev)
    idx, w = net.route(x)
    want, got = net.forward(x).double(), parts.forward(x, idx, w).double()
    # the layer's own bar against its oracle; rounding h to bf16 in front of its codes
    # (the bf16 form) moves them by up to half a step of bf16, an eighth of e4m3's
    bar = 5e-3 if quantize else 2e-2
    assert float((got - want).norm() / want.norm()) < bar
    assert parts.ops.device_status() == m.MOE_OK


def test_forward_is_the_layer_at_full_size(dev):
    net, parts = make(dev, W.FULL, 1024, kind="bias_skew")
    x = W.make_x(W.FULL, 1024, 3, "bias_skew", device=dev)
    idx, w = net.route(x)
    want, got = net.forward(x).double(), parts.forward(x, idx, w).double()
    assert float((got - want).norm() / want.norm()) < 5e-3


@pytest.mark.parametrize("quantize", [True, False])
def test_backward_stage_by_stage(dev, quantize):
    """Each stage's gradient from what the stage in front of it wrote, in 64 bits."""
    tokens = 77
    net, p = make(dev, W.TINY, tokens, quantize=quantize)
    x = W.make_x(W.TINY, tokens, 1, device=dev)
    idx, w = net.route(x)
    idx[5] = -1                                 # a token for other ranks
    idx[9, 2] = 99
    p.forward(x, idx, w)
    dy = torch.randn(x.shape, device=dev, generator=torch.Generator(dev).manual_seed(1)).bfloat16()
    dx, dw = p.backward(dy)
    kept = int(p.order.starts[-1])
    assert kept == tokens * 4 - 5 and bool((dx[5] == 0).all()) and bool((dw[5] == 0).all())
    starts = p.order.starts.tolist()

    def vals(r):
        c = (r.codes, r.scales) if quantize else R.quantise(r)
        return R.values(*c)[:kept]

    def close(got, want, mag, inner):
        err = (got.double() - want).abs()
        assert bool((err <= (132 + inner // 128) * 2.0 ** -23 * mag + 1.01 * R.BF16 * want.abs())
                    .all())
    for got, d, wt in ((p.dh, p.dout, p.w2), (p.drows, p.dgate_up, p.w13)):
        like = torch.zeros((kept, wt.inner), dtype=torch.bfloat16, device=dev)
        want, mag = R.linear(vals(d), wt.codes, wt.scales, starts, like, trans=True)
        close(got[:kept], want, mag, wt.out)
    want, mag = R.combine(p.drows, p.order.slot_of_pair)
    close(dx, want, mag, 0)
    terms = R.swiglu_grad(p.dh[:kept], p.gate_up[:kept])
    v = vals(p.dgate_up)
    assert float((v - terms).norm() / terms.norm()) < R.E4M3


def test_captured_and_replayed(dev):
    """Forward and backward as one CUDA graph, replayed with other routings and rows; the
    context's workspace is used on one stream at a time."""
    tokens = 64
    net, p = make(dev, W.TINY, tokens, quantize=False)    # the workspace takes part
    xs = [W.make_x(W.TINY, tokens, s, device=dev) for s in (1, 2, 3)]
    routes = [net.route(x) for x in xs]
    dys = [x.flip(0).contiguous() for x in xs]
    want = []
    for x, (idx, w), dy in zip(xs, routes, dys):
        y = p.forward(x, idx, w)
        want.append((y.clone(), *[t.clone() for t in p.backward(dy)]))
    x, idx, w, dy = (t.clone() for t in (xs[0], *routes[0], dys[0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.forward(x, idx, w)
        p.backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = p.forward(x, idx, w)
        dx, dw = p.backward(dy)
    for i in (2, 0, 1, 1):
        x.copy_(xs[i]), idx.copy_(routes[i][0]), w.copy_(routes[i][1]), dy.copy_(dys[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want[i]))
    assert p.ops.device_status() == m.MOE_OK


def test_large_orders_captured(dev):
    """The three launches of a large sort, replayed."""
    tokens, k = 9000, 8
    ops = m.ExpertOps(256, k, tokens, 0)
    idx = torch.randint(-3, 259, (tokens, k), device=dev, dtype=torch.int32)
    x = torch.randn((tokens, 64), device=dev).bfloat16()
    order, rows = ops.dispatch(x, idx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.dispatch(x, idx, order=order, out=rows)
    for s in range(3):
        idx.copy_(torch.randint(-3, 259, (tokens, k), device=dev, dtype=torch.int32))
        graph.replay()
        starts, pair, slot = R.order(idx, 256)
        assert torch.equal(order.slot_of_pair, slot) and torch.equal(order.starts, starts)
        kept = int(starts[-1])
        assert torch.equal(rows[:kept], x[pair[:kept].long() // k])


def test_two_contexts_on_two_streams(dev):
    tokens = 200
    nets = [make(dev, W.TINY, tokens, seed=s, quantize=False) for s in (0, 1)]
    x = W.make_x(W.TINY, tokens, 1, device=dev)
    routes = [net.route(x) for net, _ in nets]
    want = [p.forward(x, *r).clone() for (_, p), r in zip(nets, routes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in nets]
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = nets[i][1].forward(x, *routes[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_stream_given_by_hand(dev):
    ops = m.ExpertOps(1, 1, 64, 256)
    w = m.BlockWeights(torch.full((128, 256), 0x30, dtype=torch.uint8, device=dev),
                       torch.ones((1, 2), device=dev))
    x = torch.randn((64, 256), device=dev).bfloat16()
    want = ops.linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.linear(x, w, stream=s)
    s.synchronize()
    assert torch.equal(want, got)


def test_takes_the_add_norms_codes(dev):
    """A dense projection of what add_rmsnorm_quantize writes, as a block's qkv projection."""
    net, p = make(dev, W.TINY, 40)
    r, x, g = W.make_addnorm(W.TINY, 40, 1, device=dev)
    _, xn, codes, scales = net.add_rmsnorm_quantize(r, x, g, W.NORM_EPS)
    wt = m.BlockWeights(p.w13.codes[0], p.w13.scales[0])
    assert torch.equal(p.ops.linear(m.QuantRows(codes, scales), wt), p.ops.linear(xn, wt))


def test_example_runs(dev, capsys):
    P.main(tokens=200, steps=2, shape=W.TINY)
    assert "us a step" in capsys.readouterr().out


# ---- refusals ---------------------------------------------------------------

def test_refusals(dev):
    ops = m.ExpertOps(16, 2, 10, 256)
    bf = dict(dtype=torch.bfloat16, device=dev)
    idx = torch.zeros((10, 2), dtype=torch.int32, device=dev)
    x = torch.zeros((10, 256), **bf)
    order, rows = ops.dispatch(x, idx)
    w = torch.ones((10, 2), device=dev)
    wt = m.BlockWeights(torch.zeros((16, 128, 256), dtype=torch.uint8, device=dev),
                        torch.ones((16, 1, 2), device=dev))
    one = m.BlockWeights(wt.codes[0], wt.scales[0])
    other = m.ExpertOrder.empty(16, 10, 3, dev)
    for call in (
            lambda: ops.dispatch(x, idx.long()), lambda: ops.dispatch(x, idx.cpu()),
            lambda: ops.dispatch(x.float(), idx), lambda: ops.dispatch(x[:9], idx),
            lambda: ops.dispatch(x.t(), idx), lambda: ops.dispatch(x, idx[:, :1]),
            lambda: ops.dispatch(x, idx, out=rows[:19]),
            lambda: ops.dispatch(x, idx, out=rows.float()),
            lambda: ops.dispatch(x, idx, order=other),
            lambda: ops.combine(rows[:19], order, w), lambda: ops.combine(rows, other, w),
            lambda: ops.combine(rows, order, w.double()), lambda: ops.combine(rows, order, w[:9]),
            lambda: ops.combine(rows, order, w, out=x[:, :128]),
            lambda: ops.combine_grad(x[:, :128], rows, order, w),
            lambda: ops.linear(x, wt, starts=order.starts[:-1]),
            lambda: ops.linear(x, wt, starts=order.starts.long()),
            lambda: ops.linear(x[:, :128], wt, starts=order.starts),
            lambda: ops.linear(x.cpu(), one), lambda: ops.linear(x, x),
            lambda: ops.linear_grad(x, one), lambda: ops.swiglu(x[:, :255]),
            lambda: ops.swiglu_grad(x, x),
            lambda: m.QuantRows(torch.zeros((4, 256), dtype=torch.uint8, device=dev),
                                torch.zeros((4, 3), device=dev)),
            lambda: m.BlockWeights(wt.codes, wt.scales[:, :, :1])):
        with pytest.raises(ValueError):
            call()

    def status(call):
        with pytest.raises(m.MoEError) as e:
            call()
        return e.value.status
    bad, shape = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    more = torch.zeros((11, 2), dtype=torch.int32, device=dev)
    assert status(lambda: ops.dispatch(torch.zeros((11, 256), **bf), more)) == shape
    assert status(lambda: ops.linear(torch.zeros((21, 256), **bf), one)) == shape
    assert status(lambda: ops.swiglu(torch.zeros((21, 256), **bf))) == shape
    wide = m.BlockWeights(torch.zeros((16, 512), dtype=torch.uint8, device=dev),
                          torch.ones((1, 4), device=dev))
    assert status(lambda: ops.linear(torch.zeros((2, 512), **bf), wide)) == shape  # > max_width
    odd = m.BlockWeights(torch.zeros((24, 256), dtype=torch.uint8, device=dev),
                         torch.ones((1, 2), device=dev))
    assert status(lambda: ops.linear(x, odd)) == shape
    assert status(lambda: ops.linear(x, wt)) == bad                     # groups without starts
    assert status(lambda: ops.dispatch(x[:, 1:249], idx)) == bad        # not 16-byte aligned
    assert status(lambda: ops.dispatch(x[:, :252], idx)) == bad         # not whole vectors
    assert status(lambda: ops.dispatch(x[:, :248], idx, quantize=True)) == bad
    assert status(lambda: ops.combine(rows, order, w, out=rows[:10])) == bad
    assert status(lambda: ops.swiglu(rows, out=rows[:, :128])) == bad
    assert status(lambda: ops.combine_grad(x, rows, order, w, out=rows)) == bad
    assert status(lambda: ops.combine_grad(x, rows, order, w, dweights=w)) == bad
    big = torch.zeros((10, 512), **bf)
    assert status(lambda: ops.linear(big[:, :256], one, out=big[:, 128:256])) == bad
    assert ops.linear(big[:, :256], one, out=big[:, 256:384]).shape == (10, 128)
    assert ops.device_status() == m.MOE_OK


def test_refusals_of_the_c_calls(dev):
    """What the binding's own checks would stop first."""
    bad = m.MOE_ERR_INVALID_ARG
    ops = m.ExpertOps(4, 1, 8, 128)
    x = torch.zeros((8, 128), dtype=torch.bfloat16, device=dev)
    y = torch.zeros_like(x)
    idx = torch.zeros((8, 1), dtype=torch.int32, device=dev)
    order = ops.sort(idx)
    p, ref = x.data_ptr(), ctypes.byref
    rows = m.moe_rows(y.data_ptr(), 128, None, None)
    both = m.moe_rows(y.data_ptr(), 128, y.data_ptr(), y.data_ptr())
    none = m.moe_rows(None, 0, None, None)
    holes = m.moe_order(None, order.pair_of_slot.data_ptr(), order.slot_of_pair.data_ptr(), 8)
    minus = m.moe_order(order.starts.data_ptr(), order.pair_of_slot.data_ptr(),
                        order.slot_of_pair.data_ptr(), -1)
    assert m.moe_dispatch(ops.ctx, None, x, 128, 128, order._ref, ref(rows)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 128, None, ref(rows)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 128, ref(holes), ref(rows)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 128, ref(minus), ref(rows)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 128, order._ref, ref(both)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 128, order._ref, ref(none)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 128, order._ref, None) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 64, 128, order._ref, ref(rows)) == bad
    assert m.moe_dispatch(ops.ctx, idx, x, 128, 0, order._ref, ref(rows)) == bad
    assert m.moe_combine(ops.ctx, x, 128, order._ref, None, 128, y, 128) == bad
    assert m.moe_combine(ops.ctx, None, 128, order._ref, p, 128, y, 128) == bad
    w = m.BlockWeights(torch.zeros((128, 128), dtype=torch.uint8, device=dev),
                       torch.ones((1, 1), device=dev))
    xr = m.moe_rows(p, 128, None, None)
    for c in (m.moe_block_weights(None, w.scales.data_ptr(), 1, 128, 128),
              m.moe_block_weights(w.codes.data_ptr(), None, 1, 128, 128),
              m.moe_block_weights(w.codes.data_ptr() + 8, w.scales.data_ptr(), 1, 128, 128),
              m.moe_block_weights(w.codes.data_ptr(), w.scales.data_ptr(), 0, 128, 128)):
        assert m.moe_linear(ops.ctx, ref(xr), ref(c), None, 8, y, 128) == bad
    assert m.moe_linear(ops.ctx, None, w._ref, None, 8, y, 128) == bad
    assert m.moe_linear(ops.ctx, ref(xr), None, None, 8, y, 128) == bad
    assert m.moe_linear(ops.ctx, ref(xr), w._ref, None, -1, y, 128) == bad
    assert m.moe_linear(ops.ctx, ref(xr), w._ref, None, 8, None, 128) == bad
    assert m.moe_linear(ops.ctx, ref(xr), w._ref, None, 8, y, 120) == bad
    many = m.moe_block_weights(w.codes.data_ptr(), w.scales.data_ptr(), 257, 128, 128)
    assert m.moe_linear(ops.ctx, ref(xr), ref(many), idx, 8, y, 128) == \
        m.MOE_ERR_UNSUPPORTED_SHAPE
    assert m.moe_swiglu(ops.ctx, x, 128, -1, 64, ref(rows)) == bad
    assert m.moe_swiglu(ops.ctx, x, 128, 8, 0, ref(rows)) == bad
    assert m.moe_swiglu(ops.ctx, x, 128, 8, -64, ref(rows)) == bad
    assert m.moe_swiglu(ops.ctx, None, 128, 8, 64, ref(rows)) == bad
    assert m.moe_swiglu_grad(ops.ctx, None, 64, x, 128, 8, 64, ref(rows)) == bad
    assert ops.device_status() == m.MOE_OK


def test_a_bad_slot_is_reported(dev):
    ops = m.ExpertOps(4, 2, 8, 128)
    order = ops.sort(torch.zeros((8, 2), dtype=torch.int32, device=dev))
    rows = torch.ones((16, 64), dtype=torch.bfloat16, device=dev)
    order.slot_of_pair[3, 1] = 16
    y = ops.combine(rows, order, torch.ones((8, 2), device=dev))
    assert ops.device_status() == m.MOE_ERR_INVALID_ARG
    assert bool((y[[0, 1, 2, 4, 5, 6, 7]] == 2).all())
    assert ops.device_status() == m.MOE_OK
