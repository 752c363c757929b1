"""What a call returns is made under the stream that the call was given, and recorded for the
caller's own, without a GPU: stand-ins for tensors and streams note both."""
from __future__ import annotations

import contextlib

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe
from test_ops_devices import E, H, K, N, T, Stand as Base, bf16, ops, quant  # noqa: F401

OWN, GIVEN = 11, 77      # handles: the caller's current stream, the one given by hand


class Stream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, device


class Made(Base):
    """A new tensor: the stream it was made under, those it was recorded for."""

    def __init__(self, dtype, shape, on):
        super().__init__(dtype, shape, 0)
        self.on, self.recorded = on, []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)

    def zero_(self):
        return self


@pytest.fixture
def made(monkeypatch):
    """Every tensor made meanwhile."""
    at, all_ = [OWN], []

    @contextlib.contextmanager
    def under(stream):
        at.append(stream.cuda_stream)
        yield
        at.pop()

    def empty(shape, dtype=None, device=None):
        all_.append(Made(dtype, shape, at[-1]))
        return all_[-1]
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(at[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: at[-1],
                        raising=False)
    # (stand-ins are built of meta tensors, which the module's own allocations are not)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: (
        real(shape, dtype=dtype, device=device) if str(device) == "meta"
        else empty(shape, dtype, device)))
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(tuple(t.shape), t.dtype))
    return all_


def calls(ops, order, stream):  # noqa: F811
    w = moe.BlockWeights(Base(torch.uint8, (E, N, H)), Base(torch.float32, (E, 1, 1)))
    starts, weights = Base(torch.int32, (E + 1,)), Base(torch.float32, (T, K))
    idx = Base(torch.int32, (T, K))
    none = Base(torch.int32, (0, K))
    kw = dict(stream=stream)
    return {
        "sort": (3, lambda: ops.sort(idx, **kw)),
        "sort of nothing": (3, lambda: ops.sort(none, **kw)),
        "dispatch": (4, lambda: ops.dispatch(bf16(T, H), idx, **kw)),
        "dispatch to codes": (5, lambda: ops.dispatch(bf16(T, H), idx, quantize=True, **kw)),
        "dispatch_grad": (1, lambda: ops.dispatch_grad(bf16(T * K, H), order, **kw)),
        "combine": (1, lambda: ops.combine(bf16(T * K, H), order, weights, **kw)),
        "combine_grad": (2, lambda: ops.combine_grad(bf16(T, H), bf16(T * K, H), order, weights,
                                                     **kw)),
        "combine_grad to codes": (3, lambda: ops.combine_grad(
            bf16(T, H), bf16(T * K, H), order, weights, quantize=True, **kw)),
        "linear": (1, lambda: ops.linear(quant(T * K, H), w, starts=starts, **kw)),
        "linear_grad": (1, lambda: ops.linear_grad(bf16(T * K, N), w, starts=starts, **kw)),
        "swiglu": (1, lambda: ops.swiglu(bf16(T, 2 * H), **kw)),
        "swiglu to codes": (2, lambda: ops.swiglu(bf16(T, 2 * H), quantize=True, **kw)),
        "swiglu_grad": (1, lambda: ops.swiglu_grad(bf16(T, H), bf16(T, 2 * H), **kw)),
    }


@pytest.mark.parametrize("given, on, recorded", [
    (None, OWN, []), (OWN, OWN, []), (GIVEN, GIVEN, [OWN]), (0, 0, [OWN])])
def test_results_belong_to_the_stream(ops, made, given, on, recorded):  # noqa: F811
    order = moe.ExpertOrder(*[Base(torch.int32, n) for n in ((E + 1,), (T * K,), (T, K))])
    for name, (count, call) in calls(ops, order, given).items():
        made.clear()
        call()
        assert len(made) == count, name
        for t in made:
            assert t.on == on and t.recorded == recorded, name
