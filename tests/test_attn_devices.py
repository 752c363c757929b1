"""The binding's attention classes refuse tensors of another GPU than the context's, without
a GPU: the checks read dtype, device, shape and strides alone, which stand-ins have too."""
from __future__ import annotations

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe

SHAPE = moe.AttnShape(q_heads=4, kv_heads=2, head_dim=64, page_tokens=16)
ROWS = 3


class Stand:
    """What the checks see of a CUDA tensor on GPU `index` (-1: of a host tensor)."""

    def __init__(self, dtype, shape, index=0):
        self.t = torch.empty(shape, dtype=dtype, device="meta")
        self.dtype, self.shape, self.index = dtype, self.t.shape, index
        self.is_cuda = index >= 0
        self.device = torch.device("cuda", index) if self.is_cuda else torch.device("cpu")

    def get_device(self):
        return self.index

    def dim(self):
        return self.t.dim()

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def data_ptr(self):
        return 1 << 20


class Library:
    """Takes the calls that get past the checks."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def net():
    n = moe.Attention.__new__(moe.Attention)
    n.shape, n.device, n.ctx, n._lib = SHAPE, 0, None, Library()
    n._pages = (SHAPE.kv_heads, SHAPE.page_tokens, SHAPE.head_dim)
    n._gamma_shape = (SHAPE.head_dim,)
    n._at = lambda stream: 0
    return n


def cache(index=0, other=None):
    return moe.KVCache(*[Stand(torch.uint8, (5, 2, 16, 64), i) for i in (index, index)],
                       *[Stand(torch.float32, (5, 2), i)
                         for i in (index, index if other is None else other)])


def batch(index=0, other=None):
    return moe.AttnBatch(Stand(torch.int32, (2,), index), Stand(torch.int32, (1,), index),
                         Stand(torch.int32, (1, 4), index if other is None else other), ROWS)


def rows(heads, index=0):
    return Stand(torch.bfloat16, (ROWS, heads, 64), index)


def gamma(index=0):
    return Stand(torch.bfloat16, (64,), index)


def calls(net, at):
    """Every call with its tensors on GPU 0, but for the one named `at`."""
    def i(name):
        return 1 if name == at else 0
    return {
        "rope x": lambda: net.rope(rows(4, i("rope x")), Stand(torch.int32, (ROWS,)),
                                   out=rows(4)),
        "rope positions": lambda: net.rope(rows(4), Stand(torch.int32, (ROWS,),
                                                          i("rope positions")), out=rows(4)),
        "rope gamma": lambda: net.rope(rows(4), Stand(torch.int32, (ROWS,)),
                                       gamma=gamma(i("rope gamma")), out=rows(4)),
        "rope out": lambda: net.rope(rows(4), Stand(torch.int32, (ROWS,)),
                                     out=rows(4, i("rope out"))),
        "append k": lambda: net.append(rows(2, i("append k")), rows(2), cache(), batch()),
        "append v": lambda: net.append(rows(2), rows(2, i("append v")), cache(), batch()),
        "append cache": lambda: net.append(rows(2), rows(2), cache(i("append cache")), batch()),
        "append batch": lambda: net.append(rows(2), rows(2), cache(), batch(i("append batch"))),
        "forward q": lambda: net.forward(rows(4, i("forward q")), cache(), batch(), out=rows(4)),
        "forward cache": lambda: net.forward(rows(4), cache(i("forward cache")), batch(),
                                             out=rows(4)),
        "forward batch": lambda: net.forward(rows(4), cache(), batch(i("forward batch")),
                                             out=rows(4)),
        "forward out": lambda: net.forward(rows(4), cache(), batch(),
                                           out=rows(4, i("forward out"))),
        "step qkv": lambda: net.step(rows(8, i("step qkv")), cache(), batch(), out=rows(4)),
        "step cache": lambda: net.step(rows(8), cache(i("step cache")), batch(), out=rows(4)),
        "step batch": lambda: net.step(rows(8), cache(), batch(i("step batch")), out=rows(4)),
        "step q_gamma": lambda: net.step(rows(8), cache(), batch(), out=rows(4),
                                         q_gamma=gamma(i("step q_gamma"))),
        "step k_gamma": lambda: net.step(rows(8), cache(), batch(), out=rows(4),
                                         k_gamma=gamma(i("step k_gamma"))),
        "step out": lambda: net.step(rows(8), cache(), batch(), out=rows(4, i("step out"))),
    }


NAMES = list(calls(None, None))


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_of_another_gpu_is_refused(net, name):
    with pytest.raises(ValueError):
        calls(net, name)[name]()
    assert not net._lib.calls


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_the_context_s_gpu_pass(net, name):
    calls(net, None)[name]()
    assert len(net._lib.calls) == 1


@pytest.mark.parametrize("other", [1, -1])
def test_a_cache_or_a_batch_of_two_devices_is_refused(other):
    """The last of a cache's or a batch's tensors on another GPU, or on the host."""
    with pytest.raises(ValueError):
        cache(0, other)
    with pytest.raises(ValueError):
        batch(0, other)
