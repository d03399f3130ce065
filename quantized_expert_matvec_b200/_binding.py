"""ctypes binding of libqexpert.so: same entry-point names as the C ABI.

Only argument marshalling happens here; every step of the expert path runs in
the library's CUDA kernels.  Tensors must be CUDA tensors (contiguous);
``stream`` defaults to torch's current stream.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqexpert.so")

QE_OK = 0
QE_ERR_INVALID_ARG = -1
QE_ERR_UNSUPPORTED = -2
QE_ERR_CUDA = -3
QE_ERR_TIMEOUT = -4
QE_ERR_OOM = -5
QE_F32 = 0
QE_BF16 = 1
QE_F16 = 2

__all__ = [
    "LIB_PATH", "lib", "QEError", "Cfg", "QMat", "Expert", "Layer", "ExpertPool",
    "QE_OK", "QE_ERR_INVALID_ARG", "QE_ERR_UNSUPPORTED", "QE_ERR_CUDA", "QE_ERR_TIMEOUT", "QE_ERR_OOM",
    "QE_F32", "QE_BF16", "QE_F16",
    "qe_last_error", "qe_version", "qe_expert_bytes", "qe_pool_table", "qe_workspace_bytes",
    "qe_workspace_init", "qe_workspace_status", "qe_set_wait_budget_ns", "qe_test_skip_arrival", "qe_trace_fused",
    "moe_route", "moe_expert_ffn_q4", "moe_expert_ffn_q2", "moe_expert_ffn_mixed", "moe_combine",
    "moe_layer_step", "moe_layer_step_noalloc", "moe_layer_step_host", "workspace", "Tier", "TierDesc",
    "gdn_decode_step",
    "KVCache", "Rope", "attn_workspace_bytes", "attn_workspace", "attn_kv_append", "attn_decode_step", "token_sample",
]


class QEError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class Cfg(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("group", ctypes.c_int32), ("eps", ctypes.c_float)]

    def __init__(self, hidden, n_experts, top_k, inter, group=64, eps=1e-6):
        super().__init__(hidden, n_experts, top_k, inter, group, eps)


class QMat(ctypes.Structure):
    _fields_ = [("wq", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Expert(ctypes.Structure):
    _fields_ = [("gate", QMat), ("up", QMat), ("down", QMat)]


class Layer(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("logit_offset", ctypes.c_void_p), ("gamma", ctypes.c_void_p),
                ("experts", ctypes.c_void_p)]


class TierDesc(ctypes.Structure):
    _fields_ = [("cfg", Cfg), ("n_layers", ctypes.c_int32), ("cold_bits", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("cold_host", ctypes.POINTER(ctypes.c_void_p)), ("cache_bytes", ctypes.c_size_t)]


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("pair_axis", ctypes.POINTER(ctypes.c_uint8)),
                ("rotary_dim", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("adjacent", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


assert ctypes.sizeof(TierDesc) == 56
assert ctypes.sizeof(KVCacheDesc) == 56
assert ctypes.sizeof(RopeDesc) == 32


assert ctypes.sizeof(Expert) == 96


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with quantized_expert_matvec_b200/build.py "
                          "(or __graft_entry__.build()); there is no CPU fallback")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    P = ctypes.POINTER
    sigs = {
        "qe_last_error": (ctypes.c_char_p, []),
        "qe_version": (ctypes.c_char_p, []),
        "qe_expert_bytes": (sz, [P(Cfg), i32]),
        "qe_pool_table": (i32, [P(Cfg), vp, i32, i32, P(Expert), P(ctypes.c_size_t)]),
        "qe_workspace_bytes": (sz, [P(Cfg), i32]),
        "qe_workspace_init": (i32, [vp, sz, vp]),
        "qe_workspace_status": (i32, [vp, vp]),
        "qe_set_wait_budget_ns": (None, [ctypes.c_uint64]),
        "qe_test_skip_arrival": (None, [i32]),
        "qe_trace_fused": (None, [vp]),
        "moe_route": (i32, [P(Cfg), vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]),
        "moe_expert_ffn_q4": (i32, [P(Cfg), vp, vp, vp, i32, vp, vp, sz, vp]),
        "moe_expert_ffn_q2": (i32, [P(Cfg), vp, vp, vp, i32, vp, vp, sz, vp]),
        "moe_expert_ffn_mixed": (i32, [P(Cfg), vp, vp, vp, i32, vp, vp, sz, vp]),
        "moe_combine": (i32, [vp, vp, vp, i32, i32, i32, vp, vp]),
        "moe_layer_step": (i32, [P(Cfg), P(Layer), vp, i32, i32, vp, i32, vp, vp, vp, sz, vp]),
        "moe_layer_step_noalloc": (i32, [P(Cfg), P(Layer), vp, i32, vp, i32, vp, vp, vp, vp]),
        "moe_layer_step_host": (i32, [P(Cfg), P(Layer), vp, i32, i32, vp, i32, vp, sz, vp]),
        "qe_tier_create": (i32, [P(TierDesc), P(vp)]),
        "qe_tier_resolve": (i32, [vp, i32, P(ctypes.c_int32), i32, vp, vp]),
        "qe_tier_layer_step": (i32, [vp, i32, P(Layer), vp, i32, i32, vp, i32, vp, vp, vp, sz, vp]),
        "qe_tier_stats": (i32, [vp, P(ctypes.c_uint64), P(ctypes.c_uint64), P(ctypes.c_uint64)]),
        "qe_tier_slots": (i32, [vp]),
        "qe_tier_destroy": (None, [vp]),
        "gdn_decode_step": (i32, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "attn_kv_append": (i32, [P(KVCacheDesc), P(RopeDesc), i32, i32, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp, vp,
                                 vp, vp, i32, i32, vp, sz, vp]),
        "attn_workspace_bytes": (sz, [P(KVCacheDesc), i32, i32]),
        "attn_decode_step": (i32, [P(KVCacheDesc), i32, i32, vp, i64, vp, i32, vp, i32, vp, f, vp, i64, vp, vp, sz, vp]),
        "token_sample": (i32, [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != QE_OK:
        raise QEError(rc, lib.qe_last_error().decode())
    return rc


def qe_last_error() -> str:
    return lib.qe_last_error().decode()


def qe_version() -> str:
    return lib.qe_version().decode()


def qe_expert_bytes(cfg: Cfg, bits: int) -> int:
    return int(lib.qe_expert_bytes(ctypes.byref(cfg), bits))


def qe_pool_table(cfg: Cfg, base_ptr: int, bits: int, n: int):
    """Descriptors (ctypes array of Expert) and segment offsets of n experts
    stored back to back from base_ptr in the standard layout."""
    table = (Expert * max(n, 1))()
    seg = (ctypes.c_size_t * 9)()
    _check(lib.qe_pool_table(ctypes.byref(cfg), base_ptr, bits, n, table, seg))
    return table, list(seg)


def qe_workspace_bytes(cfg: Cfg, T: int) -> int:
    return int(lib.qe_workspace_bytes(ctypes.byref(cfg), T))


def qe_workspace_init(ws, stream=None):
    _check(lib.qe_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def qe_workspace_status(ws, stream=None) -> int:
    """Synchronise and return the device status (0, or a negative QE_ERR_*)."""
    return int(lib.qe_workspace_status(_ptr(ws), _stream(stream)))


def qe_set_wait_budget_ns(ns: int):
    lib.qe_set_wait_budget_ns(int(ns))


def qe_test_skip_arrival(cta: int):
    lib.qe_test_skip_arrival(int(cta))


def qe_trace_fused(buf):
    """Record per-CTA phase timestamps of fused launches into buf (uint64
    CUDA tensor [SMs, 64]); None disables."""
    lib.qe_trace_fused(_ptr(buf) if buf is not None else None)


def workspace(cfg: Cfg, T: int, device="cuda"):
    """Allocate (through torch) and zero a workspace for T tokens."""
    import torch
    n = qe_workspace_bytes(cfg, T)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    qe_workspace_init(ws)
    return ws


def _nbytes(t):
    return t.numel() * t.element_size()


def moe_route(cfg, x, gamma, router_w, logit_offset, xn, topk_idx, topk_w, ws, stream=None):
    import torch
    T = x.shape[0]
    dt = QE_BF16 if x.dtype == torch.bfloat16 else QE_F32
    _check(lib.moe_route(ctypes.byref(cfg), _ptr(x), dt, _ptr(gamma), _ptr(router_w), _ptr(logit_offset), T,
                         _ptr(xn), _ptr(topk_idx), _ptr(topk_w), _ptr(ws), _nbytes(ws), _stream(stream)))


def _ffn(fn, cfg, experts, xn, topk_idx, y, ws, stream):
    T = xn.shape[0]
    _check(fn(ctypes.byref(cfg), _ptr(experts), _ptr(xn), _ptr(topk_idx), T, _ptr(y), _ptr(ws), _nbytes(ws),
              _stream(stream)))


def moe_expert_ffn_q4(cfg, experts, xn, topk_idx, y, ws, stream=None):
    _ffn(lib.moe_expert_ffn_q4, cfg, experts, xn, topk_idx, y, ws, stream)


def moe_expert_ffn_q2(cfg, experts, xn, topk_idx, y, ws, stream=None):
    _ffn(lib.moe_expert_ffn_q2, cfg, experts, xn, topk_idx, y, ws, stream)


def moe_expert_ffn_mixed(cfg, experts, xn, topk_idx, y, ws, stream=None):
    _ffn(lib.moe_expert_ffn_mixed, cfg, experts, xn, topk_idx, y, ws, stream)


def moe_combine(y, w, residual, out, stream=None):
    T, K, H = y.shape
    _check(lib.moe_combine(_ptr(y), _ptr(w), _ptr(residual), T, K, H, _ptr(out), _stream(stream)))


def moe_layer_step(cfg, layer: Layer, x, out, add_residual=False, topk_idx=None, topk_w=None, ws=None,
                   stream=None):
    import torch
    T = x.shape[0]
    dt = QE_BF16 if x.dtype == torch.bfloat16 else QE_F32
    _check(lib.moe_layer_step(ctypes.byref(cfg), ctypes.byref(layer), _ptr(x), dt, T, _ptr(out),
                              1 if add_residual else 0, _ptr(topk_idx), _ptr(topk_w), _ptr(ws), _nbytes(ws),
                              _stream(stream)))


def moe_layer_step_noalloc(cfg, layer: Layer, x, out, add_residual=False, topk_idx=None, topk_w=None,
                           status=None, stream=None):
    """One token through the layer with the library's built-in scratch
    (no workspace, no allocation); `status` is an optional int32 device
    tensor that receives the call's device-side status."""
    import torch
    if x.shape[0] != 1:
        raise ValueError("moe_layer_step_noalloc takes exactly one token")
    dt = QE_BF16 if x.dtype == torch.bfloat16 else QE_F32
    _check(lib.moe_layer_step_noalloc(ctypes.byref(cfg), ctypes.byref(layer), _ptr(x), dt, _ptr(out),
                                      1 if add_residual else 0, _ptr(topk_idx), _ptr(topk_w), _ptr(status),
                                      _stream(stream)))


class Tier:
    """A two-tier expert store (qe_tier_*): cold_host[l][e] is the host
    address of cold expert (l, e) in the standard pool layout at cold_bits,
    or None for a hot expert.  Owns the native tier until close()."""

    def __init__(self, cfg: Cfg, cold_host, cold_bits: int, cache_bytes: int, max_tokens: int = 1):
        L = len(cold_host)
        E = cfg.n_experts
        arr = (ctypes.c_void_p * (L * E))()
        for l in range(L):
            for e in range(E):
                arr[l * E + e] = cold_host[l][e]
        self._arr = arr
        d = TierDesc(cfg, L, cold_bits, max_tokens, 0, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)),
                     int(cache_bytes))
        h = ctypes.c_void_p()
        _check(lib.qe_tier_create(ctypes.byref(d), ctypes.byref(h)))
        self.handle = h
        self.cfg = cfg

    @property
    def slots(self) -> int:
        return lib.qe_tier_slots(self.handle)

    def stats(self):
        """(hits, misses, h2d_bytes) since creation."""
        a, b, c = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
        _check(lib.qe_tier_stats(self.handle, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
        return a.value, b.value, c.value

    def resolve(self, layer: int, idx, dev_table, stream=None):
        idx = [int(i) for i in idx]
        arr = (ctypes.c_int32 * len(idx))(*idx)
        _check(lib.qe_tier_resolve(self.handle, layer, arr, len(idx), _ptr(dev_table), _stream(stream)))

    def layer_step(self, layer: int, layer_w: Layer, x, out, add_residual=False, topk_idx=None, topk_w=None,
                   ws=None, stream=None):
        import torch
        T = x.shape[0]
        dt = QE_BF16 if x.dtype == torch.bfloat16 else QE_F32
        _check(lib.qe_tier_layer_step(self.handle, layer, ctypes.byref(layer_w), _ptr(x), dt, T, _ptr(out),
                                      1 if add_residual else 0, _ptr(topk_idx), _ptr(topk_w), _ptr(ws),
                                      _nbytes(ws), _stream(stream)))

    def close(self):
        if self.handle:
            lib.qe_tier_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_layer_step_host(cfg, layer: Layer, x_host, out_host, add_residual=False, ws=None, stream=None):
    """The layer step on host tensors (pinned for asynchronous copies):
    copy in, step, copy out, synchronise."""
    import torch
    if x_host.is_cuda or out_host.is_cuda:
        raise ValueError("moe_layer_step_host takes host tensors")
    if not (x_host.is_contiguous() and out_host.is_contiguous()):
        raise ValueError("expected contiguous tensors")
    T = x_host.shape[0]
    dt = QE_BF16 if x_host.dtype == torch.bfloat16 else QE_F32
    _check(lib.moe_layer_step_host(ctypes.byref(cfg), ctypes.byref(layer), x_host.data_ptr(), dt, T,
                                   out_host.data_ptr(), 1 if add_residual else 0, _ptr(ws), _nbytes(ws),
                                   _stream(stream)))


class ExpertPool:
    """n experts of one bit width, back to back in one device buffer
    (standard layout of qe_pool_table), plus the device descriptor table."""

    def __init__(self, cfg: Cfg, n: int, bits: int, device="cuda"):
        import torch
        self.cfg, self.n, self.bits = cfg, n, bits
        self.stride = qe_expert_bytes(cfg, bits)
        if self.stride == 0:
            raise QEError(QE_ERR_INVALID_ARG, qe_last_error())
        self.buf = torch.empty(self.stride * n + 256, dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        self.base = (base + 255) // 256 * 256
        self.host_table, self.seg = qe_pool_table(cfg, self.base, bits, n)
        raw = bytes(self.host_table)[: ctypes.sizeof(Expert) * n]
        self.table = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(device)

    def seg_ptr(self, seg: int, expert: int = 0) -> int:
        """Device address of segment `seg` (0..8, qe_pool_table order) of an expert."""
        return self.base + expert * self.stride + self.seg[seg]


def gdn_decode_step(state, q, k, v, alpha, beta, out, stream=None):
    """One GatedDeltaNet decode step for every head, in place on ``state``
    (fp32 CUDA tensors: state [n_heads, dv, dk], q and k [n_heads, dk], v and
    out [n_heads, dv], alpha and beta [n_heads])."""
    import torch
    if state.dim() != 3:
        raise ValueError("state must be [n_heads, dv, dk]")
    nh, dv, dk = (int(d) for d in state.shape)
    for name, t, n in (("state", state, nh * dv * dk), ("q", q, nh * dk), ("k", k, nh * dk), ("v", v, nh * dv),
                       ("alpha", alpha, nh), ("beta", beta, nh), ("out", out, nh * dv)):
        if t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32, got {t.dtype}")
        if t.numel() != n:
            raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    _check(lib.gdn_decode_step(nh, dk, dv, _ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                               _ptr(out), _stream(stream)))


# What the attn_* and token_sample calls need of torch, looked up at their first
# use: a decode step makes these calls once a layer, and a call's host time
# counts as much as the kernel's.
_torch = _raw_stream = _device = None
_CODES = {}


def _lazy():
    global _torch, _raw_stream, _device
    import torch
    _raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _CODES.update({torch.float32: QE_F32, torch.bfloat16: QE_BF16, torch.float16: QE_F16})
    torch.cuda.current_device()  # initialises CUDA
    _torch = torch


def _code(dtype):
    try:
        return _CODES[dtype]
    except KeyError:
        raise ValueError(f"expected float32, bfloat16 or float16, got {dtype}") from None


def _placed(name, t, dtype, dev):
    """Raises for a tensor of another dtype or not on the current device."""
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _vec(name, t, dtype, n, dev):
    """Pointer of an optional dense tensor of n elements (n None: any number)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or (n is not None and t.numel() != n) or not t.is_contiguous():
        _placed(name, t, dtype, dev)
        if n is not None and t.numel() != n:
            raise ValueError(f"{name} must have {n} elements, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(name, t, dtype, T, heads, dim, dev):
    """Pointer and token stride of [T, heads, dim] with dense heads."""
    s = t.stride()
    if t.shape != (T, heads, dim) or t.get_device() != dev or t.dtype is not dtype or s[2] != 1 or (heads > 1 and s[1] != dim):
        _placed(name, t, dtype, dev)
        if t.shape != (T, heads, dim):
            raise ValueError(f"{name} must have shape {(T, heads, dim)}, got {tuple(t.shape)}")
        raise ValueError(f"the heads of {name} must be dense")
    return t.data_ptr(), s[0]


def _on(stream, dev):
    return _raw_stream(dev) if stream is None else _stream(stream)


class KVCache:
    """The paged cache of one layer over the caller's tensors: k and v
    [n_pages, n_kv, page_size, head_dim], bfloat16 or float16, each page dense
    (pages may be further apart: a slice over the layers of a larger pool)."""

    def __init__(self, k, v):
        import torch
        if _torch is None and k.is_cuda:
            _lazy()
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [n_pages, n_kv, page_size, head_dim] of one dtype and device")
        if not k.is_cuda:
            raise ValueError("expected CUDA tensors")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"the cache is bfloat16 or float16, got {k.dtype}")
        n, h, p, d = (int(x) for x in k.shape)
        for name, t in (("k", k), ("v", v)):
            if n and not t[0].is_contiguous():
                raise ValueError(f"the pages of {name} must be dense")
        page = h * p * d
        self.k, self.v, self.dtype = k, v, k.dtype
        self.n_kv, self.page_size, self.head_dim = h, p, d
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), k.stride(0) if n > 1 else page, v.stride(0) if n > 1 else page,
                                n, p, h, d, _code(k.dtype), 0)
        self._ref = ctypes.byref(self.desc)
        self._dev = k.get_device()


def _current(cache, dev):
    if cache._dev != dev:
        raise ValueError(f"the cache is on cuda:{cache._dev}, the current device is cuda:{dev}")


class Rope:
    """Rotary positions: inv_freq float32 CUDA [rotary_dim / 2]; pair_axis, the
    position axis of each pair (None: axis 0); adjacent pairs (2i, 2i + 1)
    instead of (i, i + rotary_dim / 2)."""

    def __init__(self, inv_freq, pair_axis=None, adjacent=False, n_axes=None):
        import torch
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous() or not inv_freq.is_cuda:
            raise ValueError("inv_freq must be a dense float32 CUDA vector")
        n = inv_freq.numel()
        self.inv_freq, axes = inv_freq, None
        if pair_axis is not None:
            axes = [int(i) for i in pair_axis]
            if len(axes) != n or min(axes, default=0) < 0 or max(axes, default=0) > 3:
                raise ValueError(f"pair_axis must name one of at most four axes for each of the {n} pairs")
        self.n_axes = n_axes if n_axes is not None else (max(axes, default=0) + 1 if axes else 1)
        self._axes = (ctypes.c_uint8 * n)(*axes) if axes else None
        self.desc = RopeDesc(inv_freq.data_ptr(), ctypes.cast(self._axes, ctypes.POINTER(ctypes.c_uint8)) if axes else None,
                             2 * n, self.n_axes, 1 if adjacent else 0, 0)
        self._ref = ctypes.byref(self.desc)


def attn_workspace_bytes(cache: KVCache, n_q: int, B: int) -> int:
    n = int(lib.attn_workspace_bytes(cache._ref, n_q, B))
    if n == 0:
        raise QEError(QE_ERR_INVALID_ARG, qe_last_error())
    return n


def attn_workspace(cache: KVCache, n_q: int, B: int):
    """Allocate (through torch) and zero a workspace for attn_decode_step with
    B rows of n_q heads; it serves attn_kv_append too."""
    import torch
    _current(cache, _device())
    ws = torch.empty(attn_workspace_bytes(cache, n_q, B), dtype=torch.uint8, device=cache.k.device)
    qe_workspace_init(ws)
    return ws


def attn_kv_append(cache: KVCache, q, k, v, table, kv_pos, q_out=None, rope: Rope | None = None, pos=None, seq=None,
                   ws=None, stream=None):
    """Rotate q [T, n_q, head_dim] into q_out and append k, v [T, n_kv, head_dim]
    to the cache, token t at place kv_pos[t] (int32; negative: padding) of the
    sequence whose pages are table[seq[t]] (int32 [n_seq, columns]; seq None:
    t).  pos int32 [n_axes, T] are the rotation's positions (None: kv_pos).  q may
    be None, else q_out is needed; q_out may be q itself where the dtypes agree.
    ws: any workspace."""
    if ws is None or (q_out is None and q is not None):
        raise ValueError(f"{'ws' if ws is None else 'q_out'} is missing")
    dev, D, dtype = _device(), cache.head_dim, k.dtype
    i32, T, n_kv = _torch.int32, k.shape[0], cache.n_kv
    _current(cache, dev)
    kp, ks = _heads("k", k, dtype, T, n_kv, D, dev)
    vp, vs = _heads("v", v, dtype, T, n_kv, D, dev)
    n_q, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        n_q = q.shape[1]
        qp, qs = _heads("q", q, dtype, T, n_q, D, dev)
        op, os_ = _heads("q_out", q_out, cache.dtype, T, n_q, D, dev)
    n_seq, cols = table.shape
    axes = 1
    if rope is not None:
        axes = rope.n_axes
        if rope.inv_freq.get_device() != dev:
            _placed("inv_freq", rope.inv_freq, None, dev)
    if axes > 1 and pos is not None and pos.shape[0] != axes and pos.dim() > 1:
        raise ValueError(f"pos must be [{axes}, {T}], got {tuple(pos.shape)}")
    rc = lib.attn_kv_append(cache._ref, rope._ref if rope is not None else None, T, n_q, qp, kp, vp, _code(dtype), qs, ks,
                            vs, op, os_, _vec("pos", pos, i32, axes * T, dev), _vec("kv_pos", kv_pos, i32, T, dev),
                            _vec("seq", seq, i32, T, dev), _vec("table", table, i32, None, dev), n_seq, cols,
                            _vec("ws", ws, _torch.uint8, None, dev), ws.numel(), _on(stream, dev))
    if rc:
        _check(rc)


def attn_decode_step(cache: KVCache, q, out, table, kv_len, prefix_pages=None, prefix_len=0, scale=None, lse=None,
                     ws=None, stream=None):
    """Attention of B rows q [B, n_q, head_dim] over the prefix_len tokens on
    prefix_pages (int32), shared by all rows, and each row's kv_len[b] own
    tokens on table[b] (int32 [B, columns]; kv_len negative: a padding row, left
    as it was), into out.  scale defaults to head_dim ** -0.5; lse float32
    [B, n_q] receives the logarithm of the softmax's denominator; ws is
    attn_workspace's."""
    if ws is None:
        raise ValueError("ws is missing")
    dev, D, dtype = _device(), cache.head_dim, cache.dtype
    i32 = _torch.int32
    B, n_q = q.shape[0], q.shape[1]
    _current(cache, dev)
    qp, qs = _heads("q", q, dtype, B, n_q, D, dev)
    op, os_ = _heads("out", out, dtype, B, n_q, D, dev)
    rows, cols = table.shape
    if rows != B:
        raise ValueError(f"table must have {B} rows, got {rows}")
    if prefix_len > 0 and (prefix_pages is None or prefix_pages.numel() * cache.page_size < prefix_len):
        raise ValueError("prefix_pages must hold prefix_len tokens")
    if lse is not None and lse.shape[0] != B and lse.dim() > 1:
        raise ValueError(f"lse must be [{B}, {n_q}], got {tuple(lse.shape)}")
    rc = lib.attn_decode_step(cache._ref, B, n_q, qp, qs, _vec("prefix_pages", prefix_pages, i32, None, dev), prefix_len,
                              _vec("table", table, i32, None, dev), cols, _vec("kv_len", kv_len, i32, B, dev),
                              D ** -0.5 if scale is None else scale, op, os_,
                              _vec("lse", lse, _torch.float32, B * n_q, dev), _vec("ws", ws, _torch.uint8, None, dev),
                              ws.numel(), _on(stream, dev))
    if rc:
        _check(rc)


def token_sample(logits, u, token, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None, stream=None):
    """The next token of each row of logits [B, V] from the uniform numbers u
    (float32 [B]) into token (int32 [B]): temperature, top_p, min_p float32 [B]
    and top_k int32 [B], each None for "off"; logprob float32 [B] receives the
    logarithm of the chosen token's probability among those kept."""
    if _torch is None:
        _lazy()
    dev, f32 = _device(), _torch.float32
    B, V = logits.shape
    s = logits.stride()
    if s[1] != 1 and V > 1:
        raise ValueError("logits must be [B, V] with dense rows")
    if logits.get_device() != dev:
        _placed("logits", logits, None, dev)
    rc = lib.token_sample(logits.data_ptr(), _code(logits.dtype), B, V, s[0], _vec("temperature", temperature, f32, B, dev),
                          _vec("top_k", top_k, _torch.int32, B, dev), _vec("top_p", top_p, f32, B, dev),
                          _vec("min_p", min_p, f32, B, dev), _vec("u", u, f32, B, dev),
                          _vec("token", token, _torch.int32, B, dev), _vec("logprob", logprob, f32, B, dev),
                          _on(stream, dev))
    if rc:
        _check(rc)
