"""The binding's classes of the layer's parts refuse tensors of another GPU than the
context's, and of the host, without a GPU: the checks read dtype, device, shape and strides
alone, which stand-ins have too."""
from __future__ import annotations

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe
from test_attn_devices import Library, Stand as Base

T, K, E, H, N = 5, 2, 6, 128, 64


class Stand(Base):
    def numel(self):
        return self.t.numel()


@pytest.fixture
def ops():
    o = moe.ExpertOps.__new__(moe.ExpertOps)
    o.n_experts, o.top_k, o.max_rows, o.device, o.ctx, o._lib = E, K, T, 0, None, Library()
    o._at = lambda stream: 0
    return o


def bf16(rows, width, index=0):
    return Stand(torch.bfloat16, (rows, width), index)


def quant(rows, width, index=0):
    return moe.QuantRows(Stand(torch.uint8, (rows, width), index),
                         Stand(torch.float32, (rows, -(-width // 128)), index))


def calls(ops, at, index):
    """Every call with its tensors on GPU 0, but for the one named `at`."""
    def i(name):
        return index if name == at else 0
    order = moe.ExpertOrder(*[Stand(torch.int32, n, i("order"))
                              for n in ((E + 1,), (T * K,), (T, K))]) if i("order") >= 0 else None
    w = moe.BlockWeights(Stand(torch.uint8, (E, N, H), i("w")),
                         Stand(torch.float32, (E, 1, 1), i("w"))) if i("w") >= 0 else None
    starts = Stand(torch.int32, (E + 1,), i("starts"))
    weights = Stand(torch.float32, (T, K), i("weights"))
    x = quant(T * K, H, i("codes")) if i("codes") >= 0 else None
    return {
        "dispatch": (("x", "idx", "order", "out"), lambda: ops.dispatch(
            bf16(T, H, i("x")), Stand(torch.int32, (T, K), i("idx")), order=order,
            out=bf16(T * K, H, i("out")))),
        "dispatch_grad": (("rows", "order", "out"), lambda: ops.dispatch_grad(
            bf16(T * K, H, i("rows")), order, out=bf16(T, H, i("out")))),
        "combine": (("rows", "order", "weights", "out"), lambda: ops.combine(
            bf16(T * K, H, i("rows")), order, weights, out=bf16(T, H, i("out")))),
        "combine_grad": (("dy", "rows", "order", "weights", "out", "dweights"),
                         lambda: ops.combine_grad(
            bf16(T, H, i("dy")), bf16(T * K, H, i("rows")), order, weights,
            out=bf16(T * K, H, i("out")),
            dweights=Stand(torch.float32, (T, K), i("dweights")))),
        "linear": (("codes", "w", "starts", "out"), lambda: ops.linear(
            x, w, starts=starts, out=bf16(T * K, N, i("out")))),
        "linear_grad": (("dy", "w", "starts", "out"), lambda: ops.linear_grad(
            bf16(T * K, N, i("dy")), w, starts=starts, out=bf16(T * K, H, i("out")))),
        "swiglu": (("gate_up", "out"), lambda: ops.swiglu(
            bf16(T, 2 * H, i("gate_up")), out=bf16(T, H, i("out")))),
        "swiglu_grad": (("dh", "gate_up", "out"), lambda: ops.swiglu_grad(
            bf16(T, H, i("dh")), bf16(T, 2 * H, i("gate_up")), out=bf16(T, 2 * H, i("out")))),
    }


def test_one_device_passes(ops):
    for name, (_, call) in calls(ops, None, 0).items():
        call()
        assert ops._lib.calls[-1] == "moe_" + name


def test_each_call_has_a_struct_of_its_own(ops):
    first, second = bf16(T, H), bf16(T, N)
    a, b = ops._form(first, "first"), ops._form(second, "second")
    assert a._obj is not b._obj and a._obj.stride == H and b._obj.stride == N


@pytest.mark.parametrize("index", [1, -1])
def test_other_devices_are_refused(ops, index):
    for name, (tensors, _) in calls(ops, None, 0).items():
        for at in tensors:
            if index < 0 and at in ("order", "w", "codes"):
                continue        # such objects are refused when they are made
            with pytest.raises(ValueError):
                calls(ops, at, index)[name][1]()
    assert ops._lib.calls == []


def test_objects_of_two_devices_are_refused():
    ints = [Stand(torch.int32, n, d) for n, d in (((E + 1,), 0), ((T * K,), 0), ((T, K), 1))]
    with pytest.raises(ValueError):
        moe.ExpertOrder(*ints)
    with pytest.raises(ValueError):
        moe.QuantRows(Stand(torch.uint8, (T, H), 0), Stand(torch.float32, (T, 1), 1))
    with pytest.raises(ValueError):
        moe.BlockWeights(Stand(torch.uint8, (E, N, H), 0), Stand(torch.float32, (E, 1, 1), 1))
