"""The layer's parts without a device: refusals of shapes and null arguments, the C structs'
layout, sizes."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import block_fp8_mixture_router_gb300 as moe
from block_fp8_mixture_router_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build()
    return moe.load_library()


def cfg(**kw):
    c = dict(n_experts=256, top_k=8, max_rows=1024, max_width=2048, workspace_cap_bytes=0)
    c.update(kw)
    return moe.moe_ops_config(*[c[n] for n, _ in moe.moe_ops_config._fields_])


def test_supported_shapes(lib):
    rc, n = moe.moe_ops_required_bytes(cfg())
    assert rc == moe.MOE_OK and n >= 8192 * (2048 + 64)
    for kw in (dict(n_experts=1, top_k=1, max_rows=1, max_width=0), dict(n_experts=4, top_k=16),
               dict(max_rows=65536, top_k=16, max_width=65536)):
        assert moe.moe_ops_required_bytes(cfg(**kw))[0] == moe.MOE_OK
    for kw in (dict(n_experts=0), dict(n_experts=257), dict(top_k=0), dict(top_k=17),
               dict(max_rows=0), dict(max_rows=65537), dict(max_width=-16), dict(max_width=24),
               dict(max_width=65552)):
        assert moe.moe_ops_required_bytes(cfg(**kw))[0] == moe.MOE_ERR_UNSUPPORTED_SHAPE, kw
        rc, h = moe.moe_ops_create(cfg(**kw), 0)
        assert rc == moe.MOE_ERR_UNSUPPORTED_SHAPE and not h.value
    rc, h = moe.moe_ops_create(cfg(workspace_cap_bytes=4096), 0)
    assert rc == moe.MOE_ERR_ALLOC_LIMIT and not h.value
    assert moe.moe_ops_create(cfg(), -1)[0] == moe.MOE_ERR_INVALID_ARG


def test_null_contexts(lib):
    bad = moe.MOE_ERR_INVALID_ARG
    assert moe.moe_dispatch(None, None, None, 0, 0, None, None, 0) == bad
    assert moe.moe_dispatch_grad(None, None, 0, None, 0, None, 0, 0) == bad
    assert moe.moe_combine(None, None, 0, None, None, 0, None, 0, 0) == bad
    assert moe.moe_combine_grad(None, None, 0, None, 0, None, None, 0, None, None, 0) == bad
    assert moe.moe_linear(None, None, None, None, 0, None, 0, 0) == bad
    assert moe.moe_linear_grad(None, None, None, None, 0, None, 0, 0) == bad
    assert moe.moe_swiglu(None, None, 0, 0, 0, None, 0) == bad
    assert moe.moe_swiglu_grad(None, None, 0, None, 0, 0, 0, None, 0) == bad
    assert moe.moe_ops_last_device_status(None) == bad
    moe.moe_ops_destroy(None)


def test_struct_layouts_match_the_binding(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {c: getattr(moe, c) for c in ("moe_ops_config", "moe_rows", "moe_block_weights",
                                            "moe_order")}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        for f, _ in cls._fields_:
            f = f.rstrip("_")
            lines.append(f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(ln.split()[:2]): int(ln.split()[2]) for ln in out.splitlines()}
    for name, cls in structs.items():
        assert got[(name, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(name, f.rstrip("_"))] == getattr(cls, f).offset


def test_host_tensors_are_refused():
    codes = torch.zeros((4, 256), dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.QuantRows(codes, torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        moe.BlockWeights(codes, torch.zeros((1, 2)))
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.ExpertOrder(i, i, i[None])
