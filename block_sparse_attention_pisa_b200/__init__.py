"""PISA piecewise sparse attention for NVIDIA B200 (sm_100a).

A thin ctypes binding over the C ABI in ``include/pisa.h`` (``libpisa.so``,
built in-tree by ``python -m block_sparse_attention_pisa_b200.build``). The
binding only marshals arguments: it reads shapes and device pointers from
torch tensors, allocates outputs with torch, and passes torch's current CUDA
stream. Every step of the computation runs in the library's CUDA kernels;
there is no CPU or PyTorch fallback -- if the library is missing or the
device is not a B200 the calls raise.

Besides the block-sparse path: attention under a token-exact window with its
gradient (``window_attention``, ``window_attention_backward``), and a paged cache
with the attention that reads it (``paged_cache``, ``cache_write``,
``cache_read``, ``paged_attention``).

Method: "PISA: Piecewise Sparse Attention Is Wiser for Efficient Diffusion
Transformers" (explainer of arXiv 2602.01077 on gist.science), technical
summary section 2.
"""
from __future__ import annotations

import ctypes
import os
from typing import Any, NamedTuple

ORDER_DROP, ORDER_ZERO, ORDER_FIRST, ORDER_HYBRID = -1, 0, 1, 2

__all__ = [
    "ORDER_DROP", "ORDER_ZERO", "ORDER_FIRST", "ORDER_HYBRID", "PisaError", "Shape", "HostOptions", "lib", "block_stats", "select", "attention", "attention_simt",
    "pisa", "pisa_host", "pisa_host_static", "STATIC_WORKSPACE_BYTES", "host_workspace_bytes", "head_chunks", "device_error", "num_blocks", "LIB_PATH", "SYMBOLS", "routing_norms",
    "window_attention", "window_attention_backward", "window_attention_backward_workspace", "PagedCache", "paged_cache",
    "cache_write", "cache_read", "paged_attention", "paged_attention_workspace",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpisa.so")

# entry points declared in include/pisa.h
SYMBOLS = (
    "pisa_block_stats", "pisa_select", "pisa_routing_norms", "pisa_attention", "pisa_attention_simt",
    "pisa_device_error", "pisa_status_string", "pisa_last_error", "pisa_version",
    "pisa_run_host_workspace", "pisa_run_host", "pisa_select_grouped", "pisa_run_host_static",
    "pisa_window_attention", "pisa_window_attention_backward_workspace", "pisa_window_attention_backward",
    "pisa_cache_write", "pisa_cache_read", "pisa_paged_attention_workspace", "pisa_paged_attention",
)

# PISA_STATIC_WORKSPACE_BYTES in include/pisa.h: the device region pisa_run_host_static uses
STATIC_WORKSPACE_BYTES = 32 << 20

STATUS = {0: "PISA_OK", 1: "PISA_ERR_INVALID_ARG", 2: "PISA_ERR_UNSUPPORTED",
          3: "PISA_ERR_CUDA", 4: "PISA_ERR_TIMEOUT"}


class PisaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("block", ctypes.c_int32)]


class HostOptions(ctypes.Structure):
    """pisa_host_options_t: routing weight, grouped selection and pipeline ranges (0: default)."""
    _fields_ = [("route_lambda", ctypes.c_float), ("group", ctypes.c_int32),
                ("candidates", ctypes.c_int32), ("chunks", ctypes.c_int32)]


class WindowShape(ctypes.Structure):
    """pisa_window_shape_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "N", "d")]


class Window(ctypes.Structure):
    """pisa_window_t: reach to either side (-1: no limit) and first tokens that stay visible."""
    _fields_ = [(n, ctypes.c_int32) for n in ("left", "right", "sinks")]


class CacheArgs(ctypes.Structure):
    """pisa_cache_t."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("K", "V", "k_scale", "v_scale")] +
                [(n, ctypes.c_int32) for n in ("num_pages", "Hkv", "page", "d", "type")])


class Sequences(ctypes.Structure):
    """pisa_sequences_t."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("page_table", "kv_lens", "q_lens")] +
                [(n, ctypes.c_int32) for n in ("B", "N", "max_pages")])


_lib = None


def lib():
    """The loaded ``libpisa.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m block_sparse_attention_pisa_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
    L.pisa_block_stats.argtypes = [vp, vp, Shape, i32, vp, vp, vp, vp]
    L.pisa_select.argtypes = [vp, vp, vp, f32, Shape, i32, vp, vp]
    L.pisa_select_grouped.argtypes = [vp, vp, vp, f32, Shape, i32, i32, i32, vp, vp]
    L.pisa_routing_norms.argtypes = [vp, Shape, vp, vp, vp]
    attn = [vp, vp, vp, vp, vp, vp, vp, Shape, i32, i32, f32, vp, vp]
    L.pisa_attention.argtypes = attn
    L.pisa_attention_simt.argtypes = attn
    opts = ctypes.POINTER(HostOptions)
    L.pisa_run_host_workspace.argtypes = [Shape, i32, i32, opts, ctypes.POINTER(ctypes.c_size_t)]
    L.pisa_run_host.argtypes = [vp, vp, vp, Shape, i32, i32, f32, opts, vp, ctypes.c_size_t, vp, vp]
    L.pisa_run_host_static.argtypes = [vp, vp, vp, Shape, i32, i32, f32, opts, vp, vp]
    size_p = ctypes.POINTER(ctypes.c_size_t)
    L.pisa_window_attention.argtypes = [vp, vp, vp, WindowShape, Window, f32, vp, vp, vp]
    L.pisa_window_attention_backward_workspace.argtypes = [WindowShape, Window, size_p]
    L.pisa_window_attention_backward.argtypes = [vp] * 6 + [WindowShape, Window, f32, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.pisa_cache_write.argtypes = [vp, vp, CacheArgs, Sequences, vp]
    L.pisa_cache_read.argtypes = [CacheArgs, Sequences, vp, vp, vp]
    L.pisa_paged_attention_workspace.argtypes = [CacheArgs, Sequences, i32, Window, size_p]
    L.pisa_paged_attention.argtypes = [vp, CacheArgs, Sequences, i32, Window, f32, vp, vp, vp, ctypes.c_size_t, vp]
    L.pisa_device_error.argtypes = [vp]
    L.pisa_status_string.argtypes = [ctypes.c_int]
    L.pisa_status_string.restype = ctypes.c_char_p
    L.pisa_last_error.argtypes = []
    L.pisa_last_error.restype = ctypes.c_char_p
    L.pisa_version.argtypes = []
    for name in ("pisa_block_stats", "pisa_select", "pisa_routing_norms", "pisa_attention", "pisa_attention_simt",
                 "pisa_device_error", "pisa_version", "pisa_run_host_workspace", "pisa_run_host",
                 "pisa_select_grouped", "pisa_run_host_static", "pisa_window_attention",
                 "pisa_window_attention_backward_workspace", "pisa_window_attention_backward", "pisa_cache_write",
                 "pisa_cache_read", "pisa_paged_attention_workspace", "pisa_paged_attention"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise PisaError(status, lib().pisa_last_error().decode())


def num_blocks(N: int, block: int) -> int:
    return -(-N // block)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _shape(x, block: int) -> Shape:
    if x.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous [B, H, N, d]")
    B, H, N, d = x.shape
    return Shape(B, H, N, d, block)


def _require(t, name: str, shape, dtype, device=None):
    """Raise ValueError unless ``t`` is a contiguous tensor of exactly ``shape`` and
    ``dtype`` (and, when ``device`` is given, on that CUDA device). Shapes and dtypes
    are checked first, so a wrong buffer is named before any device question."""
    import torch
    if t is None:
        raise ValueError(f"{name} is required here")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _device_of(t):
    """The CUDA device of the operands (``t`` must live on one)."""
    if not t.is_cuda:
        raise ValueError("the operands must be CUDA tensors")
    return t.device


def _stat_shapes(s: Shape, order: int):
    """(kbar / S0 shape, first-order statistic shape or None) for one order."""
    nB = num_blocks(s.N, s.block)
    kb = (s.B, s.H, nB, s.d)
    if order == ORDER_FIRST:
        return kb, (s.B, s.H, nB, s.d, s.d)
    if order == ORDER_HYBRID:
        return kb, (s.B, s.H, s.d, s.d)
    return kb, None


def _first_order_dtype(order: int):
    import torch
    return torch.bfloat16 if order == ORDER_FIRST else torch.float32


def _check_order(order: int):
    if order not in (ORDER_DROP, ORDER_ZERO, ORDER_FIRST, ORDER_HYBRID):
        raise ValueError(f"order={order} (must be -1, 0, 1 or 2)")


def block_stats(K, V, block: int, order: int = 1, out=None):
    """kbar (fp32), S0 (fp32) and the first-order statistic of every key/value block:
    per-block S1 (bf16 [B, H, nB, d, d]) at order 1, the head's Hbar (fp32
    [B, H, d, d]) at order 2, None at orders 0 and -1.
    ``out`` = (kbar, S0, S1) preallocated outputs (optional)."""
    import torch
    s = _shape(K, block)
    _check_order(order)
    nB = num_blocks(s.N, block)
    kb_shape, s1_shape = _stat_shapes(s, order)
    _require(K, "K", K.shape, torch.bfloat16)
    _require(V, "V", K.shape, torch.bfloat16)
    outs = []
    if out is not None:
        kbar, S0, S1 = out
        outs = [(kbar, "kbar", kb_shape, torch.float32), (S0, "S0", kb_shape, torch.float32)]
        if s1_shape is not None:
            outs.append((S1, "S1", s1_shape, _first_order_dtype(order)))
        else:
            S1 = None
        for t, name, shp, dt in outs:
            _require(t, name, shp, dt)
    dev = _device_of(K)
    for t, name in [(V, "V")] + [(x, n) for x, n, _, _ in outs]:
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if out is None:
        kbar = torch.empty((s.B, s.H, nB, s.d), device=K.device, dtype=torch.float32)
        S0 = torch.empty_like(kbar)
        S1 = torch.empty(s1_shape, device=K.device, dtype=_first_order_dtype(order)) if s1_shape else None
    _check(lib().pisa_block_stats(_ptr(K), _ptr(V), s, order, _ptr(kbar), _ptr(S0), _ptr(S1),
                                  _stream(K)))
    return kbar, S0, S1


def select(Q, kbar, block: int, topk: int, out=None, route=None, lam: float = 0.0,
           group: int = 1, candidates: int | None = None):
    """int32 [B, H, nB, topk]: critical blocks of every query block (ascending).
    ``route`` (fp32 [B, H, nB], from ``routing_norms``) and ``lam`` add the
    covariance term lam * M_j to every score. With ``group`` > 1 (or ``candidates``
    below nB) the selection is grouped: one proxy query per ``group`` query blocks keeps
    ``candidates`` key blocks, and each member keeps its best ``topk`` of them
    (``candidates`` = topk hands the proxy's list to every member)."""
    import torch
    s = _shape(Q, block)
    nB = num_blocks(s.N, block)
    _require(Q, "Q", Q.shape, torch.bfloat16)
    _require(kbar, "kbar", (s.B, s.H, nB, s.d), torch.float32)
    if route is not None:
        _require(route, "route", (s.B, s.H, nB), torch.float32)
    if out is not None:
        _require(out, "idx", (s.B, s.H, nB, topk), torch.int32)
    dev = _device_of(Q)
    for t, name in ((kbar, "kbar"), (route, "route"), (out, "idx")):
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    idx = (torch.empty((s.B, s.H, nB, topk), device=Q.device, dtype=torch.int32)
           if out is None else out)
    if group == 1 and (candidates is None or candidates == nB):
        _check(lib().pisa_select(_ptr(Q), _ptr(kbar), _ptr(route), float(lam), s, topk, _ptr(idx),
                                 _stream(Q)))
    else:
        cand = nB if candidates is None else int(candidates)
        _check(lib().pisa_select_grouped(_ptr(Q), _ptr(kbar), _ptr(route), float(lam), s, topk, int(group),
                                         cand, _ptr(idx), _stream(Q)))
    return idx


def routing_norms(S1, block: int, N: int, out=None):
    """(Hbar fp32 [B, H, d, d], M fp32 [B, H, nB]) from per-block bf16 S1 [B, H, nB, d, d]:
    the mean first-order matrix and each block's Frobenius deviation from it."""
    import torch
    if S1.dim() != 5 or S1.shape[-1] != S1.shape[-2]:
        raise ValueError("S1 must be [B, H, nB, d, d]")
    B, H, nB, d, _ = S1.shape
    if nB != num_blocks(N, block):
        raise ValueError("S1 block count does not match N and block")
    _require(S1, "S1", S1.shape, torch.bfloat16)
    s = Shape(B, H, N, d, block)
    if out is not None:
        Hbar, M = out
        _require(Hbar, "Hbar", (B, H, d, d), torch.float32)
        _require(M, "M", (B, H, nB), torch.float32)
    dev = _device_of(S1)
    if out is not None:
        for t, name in ((Hbar, "Hbar"), (M, "M")):
            if t.device != dev:
                raise ValueError(f"{name} is on {t.device}, expected {dev}")
    else:
        Hbar = torch.empty((B, H, d, d), device=S1.device, dtype=torch.float32)
        M = torch.empty((B, H, nB), device=S1.device, dtype=torch.float32)
    _check(lib().pisa_routing_norms(_ptr(S1), s, _ptr(Hbar), _ptr(M), _stream(S1)))
    return Hbar, M


def _attention(fn, Q, K, V, kbar, S0, S1, idx, block, order, scale, out=None):
    import torch
    s = _shape(Q, block)
    _check_order(order)
    nB = num_blocks(s.N, block)
    if idx is None or idx.dim() != 4:
        raise ValueError("idx must be an int32 [B, H, nB, topk] tensor")
    topk = int(idx.shape[-1])
    kb_shape, s1_shape = _stat_shapes(s, order)
    checks = [(Q, "Q", Q.shape, torch.bfloat16), (K, "K", Q.shape, torch.bfloat16),
              (V, "V", Q.shape, torch.bfloat16), (idx, "idx", (s.B, s.H, nB, topk), torch.int32)]
    if out is not None:
        checks.append((out, "O", Q.shape, torch.bfloat16))
    if order != ORDER_DROP:
        checks += [(kbar, "kbar", kb_shape, torch.float32), (S0, "S0", kb_shape, torch.float32)]
    if s1_shape is not None:
        checks.append((S1, "S1" if order == ORDER_FIRST else "Hbar (S1)", s1_shape, _first_order_dtype(order)))
    for t, name, shp, dt in checks:
        _require(t, name, shp, dt)
    dev = _device_of(Q)
    for t, name, _, _ in checks:
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if order == ORDER_DROP:
        kbar = S0 = S1 = None
    elif s1_shape is None:
        S1 = None
    O = torch.empty_like(Q) if out is None else out
    _check(fn(_ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(S0), _ptr(S1), _ptr(idx), s, topk,
              order, float(scale), _ptr(O), _stream(Q)))
    return O


def attention(Q, K, V, kbar, S0, S1, idx, block: int, order: int, scale: float, out=None):
    """Fused exact + Taylor attention; bf16 [B, H, N, d]. ``order``: -1 keep-or-drop,
    0 zeroth order, 1 per-block first order (S1 per block), 2 hybrid order (S1 = Hbar)."""
    return _attention(lib().pisa_attention, Q, K, V, kbar, S0, S1, idx, block, order, scale, out)


def attention_simt(Q, K, V, kbar, S0, S1, idx, block: int, order: int, scale: float, out=None):
    """The same operation on the plain CUDA-core cross-check kernel."""
    return _attention(lib().pisa_attention_simt, Q, K, V, kbar, S0, S1, idx, block, order, scale, out)


def pisa(Q, K, V, block: int, topk: int, order: int = 1, scale: float | None = None,
         route_lambda: float = 0.0, out=None, group: int = 1, candidates: int | None = None):
    """The whole path on device tensors: stats -> select -> attention. Returns (O, idx).
    With ``route_lambda`` > 0 the selection is covariance-aware: stats at order 1 ->
    routing norms -> routed select -> attention (at order 2 with the routing call's
    Hbar). ``group`` / ``candidates`` select with grouped proxies (see ``select``)."""
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    sel = dict(group=group, candidates=candidates)
    if route_lambda > 0.0:
        kbar, S0, S1 = block_stats(K, V, block, ORDER_FIRST)
        Hbar, M = routing_norms(S1, block, Q.shape[2])
        idx = select(Q, kbar, block, topk, route=M, lam=route_lambda, **sel)
        first = Hbar if order == ORDER_HYBRID else (S1 if order == ORDER_FIRST else None)
        return attention(Q, K, V, kbar, S0, first, idx, block, order, scale, out=out), idx
    kbar, S0, S1 = block_stats(K, V, block, order)
    idx = select(Q, kbar, block, topk, **sel)
    return attention(Q, K, V, kbar, S0, S1, idx, block, order, scale, out=out), idx


def head_chunks(BH: int, chunks: int):
    """Split the flattened (batch, head) axis into `chunks` contiguous ranges of near-equal size."""
    chunks = max(1, min(chunks, BH))
    edges = [BH * c // chunks for c in range(chunks + 1)]
    return [(edges[c], edges[c + 1]) for c in range(chunks) if edges[c + 1] > edges[c]]


def host_workspace_bytes(shape: Shape, topk: int, order: int, route_lambda: float = 0.0, chunks: int = 0,
                         group: int = 1, candidates: int = 0) -> int:
    """Device workspace (bytes) that ``pisa_host`` needs for this problem."""
    n = ctypes.c_size_t(0)
    o = HostOptions(float(route_lambda), int(group), int(candidates), int(chunks))
    _check(lib().pisa_run_host_workspace(shape, int(topk), int(order), ctypes.byref(o), ctypes.byref(n)))
    return int(n.value)


def pisa_host(Q, K, V, block: int, topk: int, order: int = 1, scale: float | None = None,
              device="cuda", route_lambda: float = 0.0, chunks: int = 0, out=None,
              group: int = 1, candidates: int = 0):
    """The whole path on HOST tensors [B, H, N, d] through the C ABI's ``pisa_run_host``:
    the library copies Q, K, V to the device, runs the path and copies O back, pipelined
    over ``chunks`` ranges of (batch, head) pairs (copies of one range overlap the kernels
    of another; the result equals the whole-batch device path bit for bit). Pinned host
    tensors let the copies run asynchronously. ``group`` / ``candidates`` select with
    grouped proxies as ``select`` does. Returns O on the host (``out`` if given). The
    device workspace is allocated here with torch."""
    import torch
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    s = _shape(Q, block)
    for t, name in ((Q, "Q"), (K, "K"), (V, "V")):
        _require(t, name, Q.shape, torch.bfloat16)
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor (pisa_host copies it to the device)")
    if out is None:
        out = torch.empty(Q.shape, dtype=Q.dtype, pin_memory=Q.is_pinned())
    _require(out, "O", Q.shape, torch.bfloat16)
    if out.is_cuda:
        raise ValueError("O must be a host tensor")
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    o = HostOptions(float(route_lambda), int(group), int(candidates or 0), int(chunks))
    with torch.cuda.device(dev):
        nbytes = ctypes.c_size_t(0)
        _check(lib().pisa_run_host_workspace(s, int(topk), int(order), ctypes.byref(o), ctypes.byref(nbytes)))
        ws = torch.empty(max(nbytes.value, 1), dtype=torch.uint8, device=dev)
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        _check(lib().pisa_run_host(_ptr(Q), _ptr(K), _ptr(V), s, int(topk), int(order), float(scale),
                                   ctypes.byref(o), _ptr(ws), nbytes.value, _ptr(out), stream))
    return out


def pisa_host_static(Q, K, V, block: int, topk: int, order: int = 1, scale: float | None = None,
                     device="cuda", route_lambda: float = 0.0, chunks: int = 0, out=None,
                     group: int = 1, candidates: int = 0):
    """``pisa_host`` through the C ABI's ``pisa_run_host_static``: the device workspace is
    the library's fixed region (``STATIC_WORKSPACE_BYTES`` per device) and nothing is
    allocated on the device. Calls that overlap in time on one device race on that region.
    Returns O on the host (``out`` if given, else a new host tensor)."""
    import torch
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    s = _shape(Q, block)
    for t, name in ((Q, "Q"), (K, "K"), (V, "V")):
        _require(t, name, Q.shape, torch.bfloat16)
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor (pisa_host_static copies it to the device)")
    if out is None:
        out = torch.empty(Q.shape, dtype=Q.dtype, pin_memory=Q.is_pinned())
    _require(out, "O", Q.shape, torch.bfloat16)
    if out.is_cuda:
        raise ValueError("O must be a host tensor")
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    o = HostOptions(float(route_lambda), int(group), int(candidates or 0), int(chunks))
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        _check(lib().pisa_run_host_static(_ptr(Q), _ptr(K), _ptr(V), s, int(topk), int(order), float(scale),
                                          ctypes.byref(o), _ptr(out), stream))
    return out


def _check_operands(checks):
    """The operands' CUDA device, if every (tensor, name, shape, dtype) entry is a contiguous
    tensor of its shape and dtype on it. Plain tensors that fit pass in one comparison each;
    anything else takes the checks that name what is wrong, shapes and dtypes before devices."""
    import torch
    dev = getattr(checks[0][0], "device", None)
    for t, _, shp, dt in checks:
        if not (type(t) is torch.Tensor and t.shape == shp and t.dtype is dt and t.device == dev and t.is_contiguous()):
            break
    else:
        if dev.type == "cuda":
            return dev
    for t, name, shp, dt in checks:
        _require(t, name, shp, dt)
    dev = _device_of(checks[0][0])
    for t, name, _, _ in checks:
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return dev


def _launch(fn, dev, *args):
    """fn(*args, stream) on ``dev`` (made current for the call if it is not) and its current stream."""
    import torch
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev.index)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev.index)))


def _heads(t, name: str):
    """The shape of a [B, H, N, d] operand."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a [B, H, N, d] tensor")
    return t.shape


def _window(left: int, right: int, sinks: int) -> Window:
    for x, name in ((left, "left"), (right, "right"), (sinks, "sinks")):
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name}={x} does not fit 32 bits")
    return Window(left, right, sinks)


def _workspace(t, nbytes: int, dev):
    """(address, bytes, tensor) of the caller's workspace tensor (uint8, checked) or a new one;
    the tensor has to live until the call is enqueued."""
    import torch
    if t is None:
        if nbytes == 0:
            return None, 0, None
        t = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        return t.data_ptr(), nbytes, t
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    if t.numel() < nbytes:
        raise ValueError(f"workspace holds {t.numel()} bytes, {nbytes} are needed")
    if t.device != dev:
        raise ValueError(f"workspace is on {t.device}, expected {dev}")
    return t.data_ptr(), t.numel(), t


_window_function = None


def _recorded_window_attention():
    """``window_attention`` as a torch.autograd.Function (made on first use: torch is imported late here)."""
    global _window_function
    if _window_function is None:
        import torch

        class WindowAttention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, Q, K, V, left, right, sinks, scale):
                O, lse = window_attention(Q, K, V, left, right, sinks, scale)
                ctx.save_for_backward(Q, K, V, O, lse)
                ctx.mark_non_differentiable(lse)
                ctx.call = (left, right, sinks, scale)
                return O, lse

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dO, _):
                grads = window_attention_backward(dO.contiguous(), *ctx.saved_tensors, *ctx.call)
                return *(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None, None, None

        _window_function = WindowAttention
    return _window_function


def window_attention(Q, K, V, left: int = -1, right: int = -1, sinks: int = 0, scale: float | None = None, out=None,
                     lse=None):
    """Self-attention in which the query at position p sees key j if ``j <= p + right`` and
    (``j >= p - left`` or ``j < sinks``); -1 sets no limit on a side. Q: bf16 [B, Hq, N, d];
    K, V: bf16 [B, Hkv, N, d], query head h reading key head ``h // (Hq // Hkv)``. Returns
    (O bf16 [B, Hq, N, d], lse fp32 [B, Hq, N], the natural logarithm of each row's sum). Autograd
    records the call: O carries its gradient (``window_attention_backward``'s), lse none, and
    ``out`` and ``lse`` cannot be given then. PyTorch captures a recorded backward pass only while
    no eager graph of the same leaves lives; a captured training step calls
    ``window_attention_backward`` itself."""
    import torch
    B, Hq, N, d = q = _heads(Q, "Q")
    kv, stat = (B, _heads(K, "K")[1], N, d), (B, Hq, N)
    if torch.is_grad_enabled() and (Q.requires_grad or K.requires_grad or getattr(V, "requires_grad", False)):
        if out is not None or lse is not None:
            raise ValueError("out and lse cannot be given while autograd records the call (an operand requires a gradient)")
        return _recorded_window_attention().apply(Q, K, V, left, right, sinks, scale)
    checks = [(Q, "Q", q, torch.bfloat16), (K, "K", kv, torch.bfloat16), (V, "V", kv, torch.bfloat16)]
    if out is not None:
        checks.append((out, "O", q, torch.bfloat16))
    if lse is not None:
        checks.append((lse, "lse", stat, torch.float32))
    dev = _check_operands(checks)
    O = torch.empty_like(Q) if out is None else out
    lse = Q.new_empty(stat, dtype=torch.float32) if lse is None else lse
    _launch(lib().pisa_window_attention, dev, Q.data_ptr(), K.data_ptr(), V.data_ptr(), WindowShape(B, Hq, kv[1], N, d),
            _window(left, right, sinks), d ** -0.5 if scale is None else float(scale), O.data_ptr(), lse.data_ptr())
    return O, lse


def window_attention_backward_workspace(B: int, Hq: int, Hkv: int, N: int, d: int, left: int = -1, right: int = -1,
                                        sinks: int = 0) -> int:
    """Device workspace (bytes) that ``window_attention_backward`` needs for this problem."""
    for x, name in ((B, "B"), (Hq, "Hq"), (Hkv, "Hkv"), (N, "N"), (d, "d")):
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name}={x} does not fit 32 bits")
    n = ctypes.c_size_t(0)
    _check(lib().pisa_window_attention_backward_workspace(WindowShape(B, Hq, Hkv, N, d), _window(left, right, sinks),
                                                          ctypes.byref(n)))
    return n.value


def window_attention_backward(dO, Q, K, V, O, lse, left: int = -1, right: int = -1, sinks: int = 0,
                              scale: float | None = None, out=None, workspace=None):
    """Gradients (dQ, dK, dV) of ``window_attention``'s O, from the gradient dO of O and the
    forward call's operands and results (same window and scale). ``out`` = (dQ, dK, dV)
    preallocated; ``workspace``: a uint8 tensor of at least
    ``window_attention_backward_workspace`` bytes that no other call uses meanwhile."""
    import torch
    B, Hq, N, d = q = _heads(Q, "Q")
    Hkv = _heads(K, "K")[1]
    kv, bf = (B, Hkv, N, d), torch.bfloat16
    checks = [(dO, "dO", q, bf), (Q, "Q", q, bf), (K, "K", kv, bf), (V, "V", kv, bf), (O, "O", q, bf),
              (lse, "lse", (B, Hq, N), torch.float32)]
    if out is not None:
        dQ, dK, dV = out
        checks += [(dQ, "dQ", q, bf), (dK, "dK", kv, bf), (dV, "dV", kv, bf)]
    dev = _check_operands(checks)
    ws, nbytes, hold = _workspace(workspace, window_attention_backward_workspace(B, Hq, Hkv, N, d, left, right, sinks), dev)
    if out is None:
        dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    _launch(lib().pisa_window_attention_backward, dev, dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
            lse.data_ptr(), WindowShape(B, Hq, Hkv, N, d), _window(left, right, sinks), d ** -0.5 if scale is None else float(scale),
            dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws, nbytes)
    if Hq == 0:  # keys that no query head reads
        dK.zero_(), dV.zero_()
    return dQ, dK, dV


class PagedCache(NamedTuple):
    """A paged key/value cache (pisa_cache_t): K, V [num_pages, Hkv, page, d], bf16 or
    float8_e4m3fn codes, the latter with fp32 scales [num_pages, Hkv, page]. Page size 16,
    32, 64 or 128."""
    K: Any
    V: Any
    k_scale: Any = None
    v_scale: Any = None


def paged_cache(num_pages: int, Hkv: int, page: int, d: int, dtype=None, device="cuda") -> PagedCache:
    """An empty (zeroed) cache of ``dtype`` torch.bfloat16 (default) or torch.float8_e4m3fn."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"cache dtype {dtype} (must be bfloat16 or float8_e4m3fn)")
    K, V = (torch.zeros((num_pages, Hkv, page, d), dtype=dtype, device=device) for _ in "KV")
    if dtype == torch.bfloat16:
        return PagedCache(K, V)
    return PagedCache(K, V, *(torch.zeros((num_pages, Hkv, page), dtype=torch.float32, device=device) for _ in "KV"))


def _cache_checks(cache, page_table, kv_lens, q_lens, B: int):
    """``_check_operands`` entries of a cache and its sequences."""
    import torch
    K = cache.K
    if not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise ValueError("cache K must be a [num_pages, Hkv, page, d] tensor")
    if K.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"cache K has dtype {K.dtype}, expected bfloat16 or float8_e4m3fn")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [B, max_pages] tensor")
    shape, i32 = K.shape, torch.int32
    checks = [(K, "cache K", shape, K.dtype), (cache.V, "cache V", shape, K.dtype),
              (page_table, "page_table", (B, page_table.shape[1]), i32), (kv_lens, "kv_lens", (B,), i32)]
    if K.dtype != torch.bfloat16:
        checks += [(cache.k_scale, "k_scale", shape[:3], torch.float32), (cache.v_scale, "v_scale", shape[:3], torch.float32)]
    if q_lens is not None:
        checks.append((q_lens, "q_lens", (B,), i32))
    return checks


def _cache_args(cache, page_table, kv_lens, q_lens, B: int, N: int):
    """(pisa_cache_t, pisa_sequences_t) of checked tensors."""
    import torch
    K, V, ks, vs = cache
    if K.dtype == torch.bfloat16:
        c = CacheArgs(K.data_ptr(), V.data_ptr(), None, None, *K.shape, 0)
    else:
        c = CacheArgs(K.data_ptr(), V.data_ptr(), ks.data_ptr(), vs.data_ptr(), *K.shape, 1)
    return c, Sequences(page_table.data_ptr(), kv_lens.data_ptr(), None if q_lens is None else q_lens.data_ptr(), B, N,
                        page_table.shape[1])


def cache_write(K, V, cache, page_table, kv_lens, q_lens=None):
    """Append the new tokens' keys and values (bf16 [B, Hkv, N, d]) to the cache, quantised
    as they are written if it holds 8 bits. Token t of sequence b goes to position
    ``kv_lens[b] - q_lens[b] + t`` (``kv_lens`` counts the new tokens; ``q_lens`` defaults to
    N each), in page ``page_table[b, position // page]``."""
    import torch
    B, Hkv, N, d = shape = _heads(K, "K")
    checks = [(K, "K", shape, torch.bfloat16), (V, "V", shape, torch.bfloat16)]
    dev = _check_operands(checks + _cache_checks(cache, page_table, kv_lens, q_lens, B))
    c, s = _cache_args(cache, page_table, kv_lens, q_lens, B, N)
    if c.Hkv != Hkv or c.d != d:
        raise ValueError(f"the cache holds {c.Hkv} heads of {c.d}, K has {Hkv} of {d}")
    _launch(lib().pisa_cache_write, dev, K.data_ptr(), V.data_ptr(), c, s)


def cache_read(cache, page_table, kv_lens, N: int, out=None):
    """(K, V) bf16 [B, Hkv, N, d]: the first N tokens of every sequence. Rows behind a
    sequence's last are left as they are in ``out`` = (K, V), zero without it."""
    import torch
    B = len(page_table)
    checks = _cache_checks(cache, page_table, kv_lens, None, B)
    shape = (B, cache.K.shape[1], N, cache.K.shape[3])
    if out is not None:
        K, V = out
        checks += [(K, "K", shape, torch.bfloat16), (V, "V", shape, torch.bfloat16)]
    dev = _check_operands(checks)
    if out is None:
        K, V = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in "KV")
    c, s = _cache_args(cache, page_table, kv_lens, None, B, N)
    _launch(lib().pisa_cache_read, dev, c, s, K.data_ptr(), V.data_ptr())
    return K, V


def _paged_workspace(c, s, Hq: int, w) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().pisa_paged_attention_workspace(c, s, Hq, w, ctypes.byref(n)))
    return n.value


def paged_attention_workspace(Q, cache, page_table, kv_lens, left: int = -1, right: int = 0, sinks: int = 0) -> int:
    """Device workspace (bytes) that ``paged_attention`` needs for these operands."""
    B, Hq, N, _ = _heads(Q, "Q")
    _check_operands(_cache_checks(cache, page_table, kv_lens, None, B))
    return _paged_workspace(*_cache_args(cache, page_table, kv_lens, None, B, N), Hq, _window(left, right, sinks))


def paged_attention(Q, cache, page_table, kv_lens, q_lens=None, left: int = -1, right: int = 0, sinks: int = 0,
                    scale: float | None = None, out=None, lse=None, workspace=None):
    """Attention of the new tokens Q (bf16 [B, Hq, N, d]; N = 1 for single tokens) over their
    sequences in the cache, which holds the new tokens too. Positions, ``kv_lens`` and
    ``q_lens`` as in ``cache_write``, the window as in ``window_attention`` (causal by
    default). No gradient is recorded. Returns (O bf16 [B, Hq, N, d], lse fp32 [B, Hq, N]); rows ``t >= q_lens[b]`` are
    left as they are in ``out`` and ``lse``, zero without them. ``workspace``: a uint8 tensor
    of at least ``paged_attention_workspace`` bytes that no other call uses meanwhile."""
    import torch
    B, Hq, N, d = shape = _heads(Q, "Q")
    stat = (B, Hq, N)
    checks = [(Q, "Q", shape, torch.bfloat16)]
    if out is not None:
        checks.append((out, "O", shape, torch.bfloat16))
    if lse is not None:
        checks.append((lse, "lse", stat, torch.float32))
    dev = _check_operands(checks + _cache_checks(cache, page_table, kv_lens, q_lens, B))
    c, s = _cache_args(cache, page_table, kv_lens, q_lens, B, N)
    if c.d != d:
        raise ValueError(f"the cache holds heads of {c.d}, Q has {d}")
    w = _window(left, right, sinks)
    ws, nbytes, hold = _workspace(workspace, _paged_workspace(c, s, Hq, w), dev)
    if out is None:
        out = torch.empty_like(Q) if q_lens is None else torch.zeros_like(Q)
    if lse is None:
        lse = Q.new_empty(stat, dtype=torch.float32) if q_lens is None else Q.new_zeros(stat, dtype=torch.float32)
    _launch(lib().pisa_paged_attention, dev, Q.data_ptr(), c, s, Hq, w, d ** -0.5 if scale is None else float(scale),
            out.data_ptr(), lse.data_ptr(), ws, nbytes)
    return out, lse


def device_error(stream_tensor=None):
    """Synchronise the current stream and raise if a kernel flagged the device error word."""
    import torch
    st = torch.cuda.current_stream().cuda_stream if stream_tensor is None else _stream(stream_tensor).value
    _check(lib().pisa_device_error(ctypes.c_void_p(st)))
