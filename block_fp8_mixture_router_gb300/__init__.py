"""Python binding of the block-FP8 MoE layer's C ABI (include/moe.h).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
`lib/libmoe_gb300.so`.  PyTorch provides device memory and streams.  There is
no CPU fallback: if the library is missing or fails to load, importing the
binding's entry points raises.

Low-level functions carry the C names (`moe_create`, `moe_forward`, ...) and
return the C status; `MoELayer` wraps them and raises `MoEError`.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmoe_gb300.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED_SHAPE = -2
MOE_ERR_NOT_LOADED = -3
MOE_ERR_ALLOC_LIMIT = -4
MOE_ERR_CUDA = -5
MOE_ERR_DEVICE_TIMEOUT = -6

MOE_OPT_PATH = 1
MOE_OPT_PDL = 2
MOE_OPT_POLL_LIMIT = 3
MOE_OPT_LAUNCH_EPOCH = 4
MOE_OPT_BATCH_INVARIANT = 5
MOE_OPT_ROUTER_BF16 = 6
TAG_WRAP = 0x7FFFFFFF
TAG_CLEAR = TAG_WRAP - 4096  # tags of the role-split decode kernels stay below TAG_WRAP
PATH_AUTO, PATH_DECODE, PATH_PROMPT, PATH_DECODE_CHAINED, PATH_PROMPT_MMA = 0, 1, 2, 3, 4
PATH_DECODE_ROWS = 6  # the role-split multi-row decode kernel for 2..16 rows

EXPORTED = ("moe_create", "moe_load_weights", "moe_forward", "moe_forward_host", "moe_route",
            "moe_quantize", "moe_expert_activations", "moe_set_option", "moe_required_bytes",
            "moe_last_device_status", "moe_destroy", "moe_status_string",
            "moe_profile_forward", "moe_route_static", "moe_add_rmsnorm_quantize",
            "moe_forward_codes", "moe_forward_addnorm", "moe_chain_create",
            "moe_chain_forward", "moe_chain_destroy", "moe_debug_poison_workspace",
            "moe_attn_required_bytes", "moe_attn_create", "moe_rope", "moe_kv_append",
            "moe_attn_forward", "moe_attn_step", "moe_attn_last_device_status",
            "moe_attn_destroy")

MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED = 0, 1
MOE_ROPE_PLAIN, MOE_ROPE_LINEAR, MOE_ROPE_BY_PARTS = 0, 1, 2

MOE_ROUTE_STATIC_MAX_LOGITS = 262144


class moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("inter", ctypes.c_int), ("shared_inter", ctypes.c_int),
                ("act_group", ctypes.c_int), ("max_rows", ctypes.c_int),
                ("workspace_cap_bytes", ctypes.c_size_t)]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w13", "s13", "w2", "s2", "router", "ws13", "ws2", "shared_gate")]


class moe_attn_config(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in
                 ("q_heads", "kv_heads", "head_dim", "page_tokens", "rotary_dim", "rope_layout",
                  "rope_scaling", "rope_trained_positions")] +
                [(n, ctypes.c_double) for n in
                 ("rope_base", "rope_factor", "rope_turns_low", "rope_turns_high",
                  "rope_amplitude", "softmax_scale")] +
                [(n, ctypes.c_int) for n in ("window", "max_rows", "max_seqs")] +
                [("workspace_cap_bytes", ctypes.c_size_t)])


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("n_pages", ctypes.c_int)]


class moe_attn_batch(ctypes.Structure):
    _fields_ = [("row_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("pages", ctypes.c_void_p)] + [
                    (n, ctypes.c_int) for n in
                    ("n_seqs", "pages_stride", "rows", "max_seq_rows", "max_kv_len")]


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the shared library; raises if it is missing (no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
    L = ctypes.CDLL(path)
    vp, i, ip = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)
    L.moe_create.argtypes = [ctypes.POINTER(moe_config), i, ip]
    L.moe_load_weights.argtypes = [vp, ctypes.POINTER(moe_weights), i, vp]
    L.moe_forward.argtypes = [vp, vp, vp, i, vp]
    L.moe_forward_host.argtypes = [vp, vp, vp, i, vp]
    L.moe_route.argtypes = [vp, vp, i, vp, vp, vp]
    L.moe_quantize.argtypes = [vp, vp, i, vp, vp, vp]
    L.moe_add_rmsnorm_quantize.argtypes = [vp, vp, vp, vp, ctypes.c_float, i, vp, vp, vp, vp,
                                           vp]
    L.moe_route_static.argtypes = [vp, vp, i, i, i, i, vp, vp, vp]
    L.moe_expert_activations.argtypes = [vp, i, vp, vp, vp]
    L.moe_forward_codes.argtypes = [vp, i, vp, vp, vp]
    L.moe_forward_addnorm.argtypes = [vp, vp, vp, vp, ctypes.c_float, i, vp, vp, vp, vp]
    L.moe_chain_create.argtypes = [ctypes.POINTER(ctypes.c_void_p), i, ip]
    L.moe_chain_forward.argtypes = [vp, vp, vp, i, vp]
    L.moe_chain_destroy.argtypes = [vp]
    L.moe_chain_destroy.restype = None
    L.moe_set_option.argtypes = [vp, i, i]
    L.moe_debug_poison_workspace.argtypes = [vp, i, vp]
    L.moe_profile_forward.argtypes = [vp, vp, vp, i, vp, vp, i, ctypes.POINTER(ctypes.c_int), vp]
    L.moe_required_bytes.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(ctypes.c_size_t)]
    L.moe_last_device_status.argtypes = [vp]
    L.moe_destroy.argtypes = [vp]
    L.moe_destroy.restype = None
    L.moe_status_string.argtypes = [i]
    L.moe_status_string.restype = ctypes.c_char_p
    i64, f32 = ctypes.c_int64, ctypes.c_float
    kvp, bp = ctypes.POINTER(moe_kv_cache), ctypes.POINTER(moe_attn_batch)
    L.moe_attn_required_bytes.argtypes = [ctypes.POINTER(moe_attn_config),
                                          ctypes.POINTER(ctypes.c_size_t)]
    L.moe_attn_create.argtypes = [ctypes.POINTER(moe_attn_config), i, ip]
    L.moe_rope.argtypes = [vp, vp, i64, i, vp, vp, f32, i, vp, i64, vp]
    L.moe_kv_append.argtypes = [vp, kvp, vp, i64, vp, i64, bp, vp]
    L.moe_attn_forward.argtypes = [vp, kvp, vp, i64, bp, vp, i64, vp]
    L.moe_attn_step.argtypes = [vp, kvp, vp, i64, vp, vp, f32, bp, vp, i64, vp]
    L.moe_attn_last_device_status.argtypes = [vp]
    L.moe_attn_destroy.argtypes = [vp]
    L.moe_attn_destroy.restype = None
    for n in EXPORTED:
        if n not in ("moe_destroy", "moe_status_string", "moe_chain_destroy",
                     "moe_attn_destroy"):
            getattr(L, n).restype = ctypes.c_int
    _lib = L
    return L


def status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


# ---- C names, thin wrappers (status returned as is) ------------------------

def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return ctypes.c_void_p(t.data_ptr())
    return ctypes.c_void_p(int(t))


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def moe_create(cfg: moe_config, device: int = 0):
    h = ctypes.c_void_p()
    rc = load_library().moe_create(ctypes.byref(cfg), device, ctypes.byref(h))
    return rc, h


def moe_load_weights(ctx, w: moe_weights, pointers_on_device: int, stream=None) -> int:
    return load_library().moe_load_weights(ctx, ctypes.byref(w), pointers_on_device,
                                           _stream(stream))


def moe_forward(ctx, x, y, rows: int, stream=None) -> int:
    return load_library().moe_forward(ctx, _ptr(x), _ptr(y), rows, _stream(stream))


def moe_forward_host(ctx, x, y, rows: int, stream=None) -> int:
    return load_library().moe_forward_host(ctx, _ptr(x), _ptr(y), rows, _stream(stream))


def moe_debug_poison_workspace(ctx, byte: int, stream=None) -> int:
    """Fills the context's data workspace with `byte` (a test of the
    kernels' independence from earlier calls' leftovers)."""
    return load_library().moe_debug_poison_workspace(ctx, byte, _stream(stream))


def moe_route(ctx, x, rows: int, idx, w, stream=None) -> int:
    return load_library().moe_route(ctx, _ptr(x), rows, _ptr(idx), _ptr(w), _stream(stream))


def moe_route_static(x, router, rows: int, hidden: int, n_experts: int, top_k: int, idx, w,
                     stream=None) -> int:
    """The router on the library's fixed scratch (allocates nothing); calls on
    one device must not overlap."""
    return load_library().moe_route_static(_ptr(x), _ptr(router), rows, hidden, n_experts,
                                           top_k, _ptr(idx), _ptr(w), _stream(stream))


def moe_quantize(ctx, x, rows: int, codes, scales, stream=None) -> int:
    return load_library().moe_quantize(ctx, _ptr(x), rows, _ptr(codes), _ptr(scales),
                                       _stream(stream))


def moe_add_rmsnorm_quantize(ctx, residual, x, gamma, eps: float, rows: int, h_out, xn_out,
                             codes, scales, stream=None) -> int:
    return load_library().moe_add_rmsnorm_quantize(
        ctx, _ptr(residual), _ptr(x), _ptr(gamma), float(eps), rows, _ptr(h_out), _ptr(xn_out),
        _ptr(codes), _ptr(scales), _stream(stream))


def moe_expert_activations(ctx, rows: int, hq, sh, stream=None) -> int:
    return load_library().moe_expert_activations(ctx, rows, _ptr(hq), _ptr(sh), _stream(stream))


def moe_forward_addnorm(ctx, residual, x, gamma, eps: float, rows: int, h_out, xn_out, y,
                        stream=None) -> int:
    return load_library().moe_forward_addnorm(ctx, _ptr(residual), _ptr(x), _ptr(gamma),
                                              float(eps), rows, _ptr(h_out), _ptr(xn_out),
                                              _ptr(y), _stream(stream))


def moe_chain_create(ctxs):
    arr = (ctypes.c_void_p * len(ctxs))(*[c.value if isinstance(c, ctypes.c_void_p) else c
                                          for c in ctxs])
    h = ctypes.c_void_p()
    rc = load_library().moe_chain_create(arr, len(ctxs), ctypes.byref(h))
    return rc, h


def moe_chain_forward(chain, x, y_all, rows: int, stream=None) -> int:
    return load_library().moe_chain_forward(chain, _ptr(x), _ptr(y_all), rows, _stream(stream))


def moe_chain_destroy(chain) -> None:
    load_library().moe_chain_destroy(chain)


def moe_forward_codes(ctx, rows: int, codes, scales, stream=None) -> int:
    return load_library().moe_forward_codes(ctx, rows, _ptr(codes), _ptr(scales),
                                            _stream(stream))


def moe_profile_forward(ctx, x, y, rows: int, stream=None, capacity: int = 16):
    """-> (status, [(stage name, device ms), ...])"""
    ms = (ctypes.c_float * capacity)()
    names = (ctypes.c_char_p * capacity)()
    n = ctypes.c_int()
    rc = load_library().moe_profile_forward(ctx, _ptr(x), _ptr(y), rows, ctypes.cast(ms, ctypes.c_void_p),
                                            ctypes.cast(names, ctypes.c_void_p), capacity,
                                            ctypes.byref(n), _stream(stream))
    return rc, [(names[i].decode(), float(ms[i])) for i in range(n.value)]


def moe_attn_required_bytes(cfg: moe_attn_config):
    n = ctypes.c_size_t()
    rc = load_library().moe_attn_required_bytes(ctypes.byref(cfg), ctypes.byref(n))
    return rc, n.value


def moe_attn_create(cfg: moe_attn_config, device: int = 0):
    h = ctypes.c_void_p()
    rc = load_library().moe_attn_create(ctypes.byref(cfg), device, ctypes.byref(h))
    return rc, h


def moe_rope(ctx, x, x_stride: int, heads: int, positions, gamma, eps: float, rows: int, y,
             y_stride: int, stream=None) -> int:
    return load_library().moe_rope(ctx, _ptr(x), x_stride, heads, _ptr(positions), _ptr(gamma),
                                   eps, rows, _ptr(y), y_stride, _stream(stream))


def moe_kv_append(ctx, cache, k, k_stride: int, v, v_stride: int, batch, stream=None) -> int:
    """cache: a moe_kv_cache, batch: a moe_attn_batch (each may be None)."""
    return load_library().moe_kv_append(ctx, cache, _ptr(k), k_stride, _ptr(v), v_stride, batch,
                                        _stream(stream))


def moe_attn_forward(ctx, cache, q, q_stride: int, batch, out, out_stride: int,
                     stream=None) -> int:
    return load_library().moe_attn_forward(ctx, cache, _ptr(q), q_stride, batch, _ptr(out),
                                           out_stride, _stream(stream))


def moe_attn_step(ctx, cache, qkv, qkv_stride: int, q_gamma, k_gamma, eps: float, batch, out,
                  out_stride: int, stream=None) -> int:
    return load_library().moe_attn_step(ctx, cache, _ptr(qkv), qkv_stride, _ptr(q_gamma),
                                        _ptr(k_gamma), eps, batch, _ptr(out), out_stride,
                                        _stream(stream))


def moe_attn_last_device_status(ctx) -> int:
    return load_library().moe_attn_last_device_status(ctx)


def moe_attn_destroy(ctx) -> None:
    load_library().moe_attn_destroy(ctx)


def moe_set_option(ctx, option: int, value: int) -> int:
    return load_library().moe_set_option(ctx, option, value)


def moe_required_bytes(cfg: moe_config):
    n = ctypes.c_size_t()
    rc = load_library().moe_required_bytes(ctypes.byref(cfg), ctypes.byref(n))
    return rc, n.value


def moe_last_device_status(ctx) -> int:
    return load_library().moe_last_device_status(ctx)


def moe_destroy(ctx) -> None:
    load_library().moe_destroy(ctx)


def moe_status_string(status: int) -> str:
    return status_string(status)


# ---- convenience wrapper ---------------------------------------------------

@dataclass
class LayerShape:
    hidden: int = 2048
    n_experts: int = 256
    top_k: int = 8
    inter: int = 512
    shared_inter: int = 512
    act_group: int = 128


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoEError(rc, what)


class MoELayer:
    """One layer on one GPU: owns a context, its device weights and workspace."""

    def __init__(self, shape: LayerShape, max_rows: int = 1024, device: int = 0,
                 workspace_cap_bytes: int = 0):
        self.shape = shape
        self.max_rows = max_rows
        self.device = device
        cfg = moe_config(shape.hidden, shape.n_experts, shape.top_k, shape.inter,
                         shape.shared_inter, shape.act_group, max_rows, workspace_cap_bytes)
        rc, h = moe_create(cfg, device)
        _check(rc, "moe_create")
        self.ctx = h

    def close(self):
        if getattr(self, "ctx", None):
            moe_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load(self, layer: dict, stream=None):
        """Weights as torch tensors (see include/moe.h for names, dtypes, layouts)."""
        names = ("w13", "s13", "w2", "s2", "router", "ws13", "ws2", "shared_gate")
        ts = [layer[n].contiguous() for n in names]
        on_dev = {t.is_cuda for t in ts}
        if len(on_dev) != 1:
            raise ValueError("weights must be all on the device or all on the host")
        w = moe_weights(*[t.data_ptr() for t in ts])
        _check(moe_load_weights(self.ctx, w, 1 if ts[0].is_cuda else 0, stream),
               "moe_load_weights")
        self._keep = ts  # alive until the synchronous copy returned

    def set_option(self, option: int, value: int):
        _check(moe_set_option(self.ctx, option, value), "moe_set_option")

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2:
            raise ValueError("x must be a 2-D bf16 CUDA tensor")
        x = x.contiguous()
        if y is None:
            y = torch.empty_like(x)
        _check(moe_forward(self.ctx, x, y, x.shape[0], stream), "moe_forward")
        return y

    def forward_addnorm(self, residual: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor,
                        eps: float, keep_xn: bool = False, stream=None):
        """Residual add + RMS norm + the layer: returns (h, xn or None, y)."""
        for t in (residual, x, gamma):
            if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("residual, x and gamma must be contiguous bf16 CUDA tensors")
        T, H = x.shape
        h = torch.empty_like(x)
        xn = torch.empty_like(x) if keep_xn else None
        y = torch.empty_like(x)
        _check(moe_forward_addnorm(self.ctx, residual, x, gamma, eps, T, h, xn, y, stream),
               "moe_forward_addnorm")
        return h, xn, y

    def forward_host(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None):
        if x.dtype != torch.bfloat16 or x.is_cuda:
            raise ValueError("x must be a host bf16 tensor")
        if y is None:
            y = torch.empty_like(x)
        _check(moe_forward_host(self.ctx, x, y, x.shape[0], stream), "moe_forward_host")
        return y

    def poison_workspace(self, byte: int = 0xFF, stream=None):
        _check(moe_debug_poison_workspace(self.ctx, byte, stream), "moe_debug_poison_workspace")

    def route(self, x: torch.Tensor, stream=None):
        T = x.shape[0]
        idx = torch.empty((T, self.shape.top_k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, self.shape.top_k), dtype=torch.float32, device=x.device)
        _check(moe_route(self.ctx, x.contiguous(), T, idx, w, stream), "moe_route")
        return idx, w

    def quantize(self, x: torch.Tensor, stream=None):
        T, H = x.shape
        codes = torch.empty((T, H), dtype=torch.uint8, device=x.device)
        scales = torch.empty((T, H // 128), dtype=torch.float32, device=x.device)
        _check(moe_quantize(self.ctx, x.contiguous(), T, codes, scales, stream), "moe_quantize")
        return codes, scales

    def add_rmsnorm_quantize(self, residual: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor,
                             eps: float, h_out=None, xn_out=None, stream=None):
        """Residual add + RMS norm + the normed rows' FP8 groups, one launch.
        Returns (h, xn, codes, scales); h_out / xn_out may be `residual` or `x`
        for an in-place update."""
        for t in (residual, x, gamma):
            if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("residual, x and gamma must be contiguous bf16 CUDA tensors")
        T, H = x.shape
        if residual.shape != x.shape or gamma.shape != (H,):
            raise ValueError("residual and x must be [rows, H] and gamma [H]")
        h_out = torch.empty_like(x) if h_out is None else h_out
        xn_out = torch.empty_like(x) if xn_out is None else xn_out
        codes = torch.empty((T, H), dtype=torch.uint8, device=x.device)
        scales = torch.empty((T, H // 128), dtype=torch.float32, device=x.device)
        _check(moe_add_rmsnorm_quantize(self.ctx, residual, x, gamma, eps, T, h_out, xn_out,
                                        codes, scales, stream), "moe_add_rmsnorm_quantize")
        return h_out, xn_out, codes, scales

    def expert_activations(self, rows: int, stream=None):
        k, I = self.shape.top_k, self.shape.inter
        dev = torch.device("cuda", self.device)
        hq = torch.empty((rows, k, I), dtype=torch.uint8, device=dev)
        sh = torch.empty((rows, k, I // 128), dtype=torch.float32, device=dev)
        _check(moe_expert_activations(self.ctx, rows, hq, sh, stream), "moe_expert_activations")
        return hq, sh

    def forward_codes(self, rows: int, stream=None):
        """The e4m3 codes and group scales of x that the experts of the most
        recent forward read: ([rows, k, H] uint8, [rows, k, H/128] fp32)."""
        k, H = self.shape.top_k, self.shape.hidden
        dev = torch.device("cuda", self.device)
        codes = torch.empty((rows, k, H), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, k, H // 128), dtype=torch.float32, device=dev)
        _check(moe_forward_codes(self.ctx, rows, codes, scales, stream), "moe_forward_codes")
        return codes, scales

    def profile(self, x: torch.Tensor, y: torch.Tensor, stream=None):
        rc, stages = moe_profile_forward(self.ctx, x, y, x.shape[0], stream)
        _check(rc, "moe_profile_forward")
        return stages

    def device_status(self) -> int:
        return moe_last_device_status(self.ctx)


class MoEChain:
    """Layers in sequence (each a MoELayer that must outlive the chain): the
    output of layer l is the input of layer l + 1."""

    def __init__(self, layers):
        self.layers = list(layers)
        rc, h = moe_chain_create([net.ctx for net in self.layers])
        _check(rc, "moe_chain_create")
        self.chain = h

    def close(self):
        if getattr(self, "chain", None):
            moe_chain_destroy(self.chain)
            self.chain = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x: torch.Tensor, y_all: torch.Tensor | None = None, stream=None):
        """x [rows, H] bf16 -> every layer's output [n_layers, rows, H]."""
        if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2:
            raise ValueError("x must be a 2-D bf16 CUDA tensor")
        x = x.contiguous()
        if y_all is None:
            y_all = torch.empty((len(self.layers),) + tuple(x.shape), dtype=x.dtype,
                                device=x.device)
        _check(moe_chain_forward(self.chain, x, y_all, x.shape[0], stream), "moe_chain_forward")
        return y_all


# ---- attention over an 8-bit paged cache -----------------------------------

_ROPE_LAYOUTS = {"half": MOE_ROPE_HALF, "interleaved": MOE_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"plain": MOE_ROPE_PLAIN, "linear": MOE_ROPE_LINEAR,
                  "by_parts": MOE_ROPE_BY_PARTS}


@dataclass
class AttnShape:
    """An attention layer's shape (moe_attn_config in include/moe.h)."""
    q_heads: int = 16
    kv_heads: int = 2
    head_dim: int = 128
    page_tokens: int = 64
    rotary_dim: int = 128
    rope_layout: str = "half"        # half | interleaved
    rope_base: float = 10000.0
    rope_scaling: str = "plain"      # plain | linear | by_parts
    rope_factor: float = 1.0
    rope_trained_positions: int = 0
    rope_turns_low: float = 0.0
    rope_turns_high: float = 0.0
    rope_amplitude: float = 1.0
    softmax_scale: float = 0.0       # 0: 1 / sqrt(head_dim)
    window: int = 0                  # 0: all earlier positions

    def config(self, max_rows: int, max_seqs: int, workspace_cap_bytes: int = 0):
        if self.rope_layout not in _ROPE_LAYOUTS or self.rope_scaling not in _ROPE_SCALINGS:
            raise ValueError("unknown rope_layout or rope_scaling")
        return moe_attn_config(
            self.q_heads, self.kv_heads, self.head_dim, self.page_tokens, self.rotary_dim,
            _ROPE_LAYOUTS[self.rope_layout], _ROPE_SCALINGS[self.rope_scaling],
            self.rope_trained_positions, self.rope_base, self.rope_factor, self.rope_turns_low,
            self.rope_turns_high, self.rope_amplitude, self.softmax_scale, self.window, max_rows,
            max_seqs, workspace_cap_bytes)


class KVCache:
    """One layer's paged cache: e4m3 codes [pages][kv_heads][page_tokens][head_dim]
    (uint8) and fp32 scales [pages][kv_heads], for keys and for values."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.device = k_codes.get_device()
        for t, kind, dims in ((k_codes, torch.uint8, 4), (v_codes, torch.uint8, 4),
                              (k_scales, torch.float32, 2), (v_scales, torch.float32, 2)):
            if t.dtype != kind or not t.is_cuda or t.get_device() != self.device or \
                    not t.is_contiguous() or t.dim() != dims:
                raise ValueError("codes must be contiguous 4-D uint8 and scales contiguous 2-D "
                                 "fp32 CUDA tensors of one device")
        if k_codes.shape != v_codes.shape or k_scales.shape != v_scales.shape or \
                k_scales.shape != k_codes.shape[:2]:
            raise ValueError("keys and values, codes and scales must agree in shape")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = \
            k_codes, v_codes, k_scales, v_scales
        self._c = moe_kv_cache(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                               v_scales.data_ptr(), k_codes.shape[0])
        self._ref = ctypes.byref(self._c)
        self._pages = tuple(k_codes.shape[1:])

    @classmethod
    def empty(cls, shape: AttnShape, n_pages: int, device="cuda"):
        """A cache of unwritten pages."""
        def codes():
            return torch.empty((n_pages, shape.kv_heads, shape.page_tokens, shape.head_dim),
                               dtype=torch.uint8, device=device)

        def scales():
            return torch.empty((n_pages, shape.kv_heads), dtype=torch.float32, device=device)
        return cls(codes(), codes(), scales(), scales())


class AttnBatch:
    """The rows of one call (moe_attn_batch): int32 CUDA tensors row_start
    [n_seqs + 1], kv_len [n_seqs] (with this call's rows) and pages [n_seqs][most pages].
    Their contents may change from call to call (a captured graph replays with new
    lengths); max_seq_rows and max_kv_len bound them for the launch's sake."""

    def __init__(self, row_start, kv_len, pages, rows: int, max_seq_rows: int = 0,
                 max_kv_len: int = 0):
        self.device = row_start.get_device()
        for t, dims in ((row_start, 1), (kv_len, 1), (pages, 2)):
            if t.dtype != torch.int32 or not t.is_cuda or t.get_device() != self.device or \
                    t.dim() != dims or not t.is_contiguous():
                raise ValueError("row_start, kv_len and pages must be contiguous int32 CUDA "
                                 "tensors of 1, 1 and 2 dimensions, of one device")
        n = kv_len.shape[0]
        if row_start.shape[0] != n + 1 or pages.shape[0] != n:
            raise ValueError("row_start has one entry more than kv_len, pages one row for each")
        self.row_start, self.kv_len, self.pages, self.rows = row_start, kv_len, pages, rows
        self._c = moe_attn_batch(row_start.data_ptr(), kv_len.data_ptr(), pages.data_ptr(), n,
                                 pages.shape[1], rows, max_seq_rows, max_kv_len)
        self._ref = ctypes.byref(self._c)


def _rows3(t: torch.Tensor, rows: int, heads: int, dim: int, what: str, device: int) -> int:
    """Row stride of a [rows, heads, dim] bf16 tensor of a GPU whose heads lie side by side.
    (A host tensor's device number is -1.)"""
    if t.dtype is not torch.bfloat16 or t.get_device() != device or t.shape != (rows, heads, dim):
        raise ValueError(f"{what} must be a bf16 tensor [{rows}, {heads}, {dim}] of CUDA device "
                         f"{device}")
    sr, sh, sd = t.stride()
    if (sd != 1 and rows) or (sh != dim and heads > 1 and rows):
        raise ValueError(f"{what}: the heads of a row must lie side by side")
    return sr if rows > 1 else heads * dim


class Attention:
    """The attention of one layer shape on one GPU: owns a context and its workspace."""

    def __init__(self, shape: AttnShape, max_rows: int = 1024, max_seqs: int = 1,
                 device: int = 0, workspace_cap_bytes: int = 0):
        self.shape = shape
        self.device = device
        rc, h = moe_attn_create(shape.config(max_rows, max_seqs, workspace_cap_bytes), device)
        _check(rc, "moe_attn_create")
        self.ctx = h
        self._lib = load_library()
        self._pages = (shape.kv_heads, shape.page_tokens, shape.head_dim)
        self._gamma_shape = (shape.head_dim,)

    def close(self):
        if getattr(self, "ctx", None):
            moe_attn_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _at(self, stream) -> int:
        """The stream's handle; None: PyTorch's current stream of the device."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)

    def _cache_ok(self, cache: KVCache, batch: AttnBatch):
        if cache._pages != self._pages:
            raise ValueError("the cache's pages are not of this shape")
        if cache.device != self.device or batch.device != self.device:
            raise ValueError(f"the cache and the batch must be of CUDA device {self.device}")

    def _gamma(self, g):
        if g is None:
            return None
        if g.dtype is not torch.bfloat16 or g.get_device() != self.device or \
                g.shape != self._gamma_shape or not g.is_contiguous():
            raise ValueError(f"a gamma must be a contiguous bf16 tensor [head_dim] of CUDA device "
                             f"{self.device}")
        return g.data_ptr()

    def _out(self, like, rows):
        return torch.empty((rows, self.shape.q_heads, self.shape.head_dim), dtype=torch.bfloat16,
                           device=like.device)

    def rope(self, x: torch.Tensor, positions: torch.Tensor, gamma: torch.Tensor | None = None,
             eps: float = 1e-6, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Rotary positions of x [rows, heads, head_dim] (queries or keys, any number of
        heads), after an RMS norm of each head where gamma is given; out may be x."""
        if x.dim() != 3:
            raise ValueError("x must be [rows, heads, head_dim]")
        rows, heads, dim = x.shape[0], x.shape[1], self.shape.head_dim
        xs = _rows3(x, rows, heads, dim, "x", self.device)
        if positions.dtype is not torch.int32 or positions.get_device() != self.device or \
                positions.shape != (rows,) or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 tensor [rows] of CUDA device "
                             f"{self.device}")
        if out is None:
            out = torch.empty((rows, heads, dim), dtype=torch.bfloat16, device=x.device)
        rc = self._lib.moe_rope(self.ctx, x.data_ptr(), xs, heads, positions.data_ptr(),
                                self._gamma(gamma), eps, rows, out.data_ptr(),
                                _rows3(out, rows, heads, dim, "out", self.device), self._at(stream))
        if rc:
            raise MoEError(rc, "moe_rope")
        return out

    def append(self, k: torch.Tensor, v: torch.Tensor, cache: KVCache, batch: AttnBatch,
               stream=None):
        """Rows of keys and values [rows, kv_heads, head_dim] into the cache."""
        s, n = self.shape, batch.rows
        ks = _rows3(k, n, s.kv_heads, s.head_dim, "k", self.device)
        vs = _rows3(v, n, s.kv_heads, s.head_dim, "v", self.device)
        self._cache_ok(cache, batch)
        rc = self._lib.moe_kv_append(self.ctx, cache._ref, k.data_ptr(), ks, v.data_ptr(), vs,
                                     batch._ref, self._at(stream))
        if rc:
            raise MoEError(rc, "moe_kv_append")

    def forward(self, q: torch.Tensor, cache: KVCache, batch: AttnBatch,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of q [rows, q_heads, head_dim] over the cache, which already
        holds the batch's rows."""
        s, n = self.shape, batch.rows
        qs = _rows3(q, n, s.q_heads, s.head_dim, "q", self.device)
        if out is None:
            out = self._out(q, n)
        self._cache_ok(cache, batch)
        rc = self._lib.moe_attn_forward(self.ctx, cache._ref, q.data_ptr(), qs, batch._ref,
                                        out.data_ptr(),
                                        _rows3(out, n, s.q_heads, s.head_dim, "out", self.device),
                                        self._at(stream))
        if rc:
            raise MoEError(rc, "moe_attn_forward")
        return out

    def step(self, qkv: torch.Tensor, cache: KVCache, batch: AttnBatch,
             q_gamma: torch.Tensor | None = None, k_gamma: torch.Tensor | None = None,
             eps: float = 1e-6, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The whole attention step from a projection's rows [rows, q_heads + 2 kv_heads,
        head_dim]: norms and rotates, appends, attends."""
        s, n = self.shape, batch.rows
        xs = _rows3(qkv, n, s.q_heads + 2 * s.kv_heads, s.head_dim, "qkv", self.device)
        if out is None:
            out = self._out(qkv, n)
        self._cache_ok(cache, batch)
        rc = self._lib.moe_attn_step(self.ctx, cache._ref, qkv.data_ptr(), xs,
                                     self._gamma(q_gamma), self._gamma(k_gamma), eps, batch._ref,
                                     out.data_ptr(),
                                     _rows3(out, n, s.q_heads, s.head_dim, "out", self.device),
                                     self._at(stream))
        if rc:
            raise MoEError(rc, "moe_attn_step")
        return out

    def device_status(self) -> int:
        return moe_attn_last_device_status(self.ctx)
