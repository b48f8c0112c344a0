"""Binding of libmoe.so (include/moe.h). Argument marshalling only: device
tensors are passed as raw pointers with the caller's current HIP stream; every
computation runs in the library's kernels. The layer's calls go through
ctypes; those of the operators beside it through _tensors.so, which refuses
tensors that do not fit the call's description. There is no fallback: if a
library is missing the import of a call fails loudly."""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")
TENSORS_PATH = os.path.join(HERE, "_tensors.so")

MOE_STATUS_MISS = 1
MOE_STATUS_NAN_KEY = 2
MOE_STATUS_BAD_PICK = 4
MOE_K_GATEUP, MOE_K_DOWN, MOE_K_ROUTER, MOE_K_SHARED_GU, MOE_K_SHARED_DOWN, MOE_K_GATEUP2, MOE_K_DOWN2 = (
    1, 2, 3, 4, 5, 6, 7)
MOE_K_READ_PROBE = 8


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmoe error {code}: {msg}")
        self.code = code


class Cfg(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_routed", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("norm_topk_prob", ctypes.c_int32), ("gate_temp", ctypes.c_float),
                ("route_scale", ctypes.c_float), ("swiglu_limit", ctypes.c_float), ("score_mode", ctypes.c_int32)]


class Experts(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("stride", ctypes.c_uint64), ("gate_off", ctypes.c_uint64),
                ("up_off", ctypes.c_uint64), ("down_off", ctypes.c_uint64)]


class Layer(ctypes.Structure):
    _fields_ = [("gate_w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("experts", Experts),
                ("sh_w1", ctypes.c_void_p), ("sh_w3", ctypes.c_void_p), ("sh_w2", ctypes.c_void_p),
                ("shared_kind", ctypes.c_int32), ("shared_q", Experts)]


MOE_SHARED_BF16, MOE_SHARED_KQUANT = 0, 1


class CacheStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("hits", "misses", "prefetched", "prefetch_used", "bytes_copied",
                                               "reads_back")]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("total", "xq", "xd", "xs", "logits", "scores", "plan", "g", "u",
                                                 "h", "hq", "hd", "hs", "y", "sg", "su", "sh", "sd", "yr",
                                                 "status", "ctl", "grp", "xd64", "hd64")] + [("max_pairs", ctypes.c_int32),
                                                               ("plan_words", ctypes.c_int32)]


_lib = None
_VP = ctypes.c_void_p


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built: run __graft_entry__.build() (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_header_words.restype = ctypes.c_int32
        L.moe_header_words.argtypes = [ctypes.POINTER(Cfg)]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_workspace_bytes.argtypes = [ctypes.POINTER(Cfg), ctypes.c_int32]
        L.moe_workspace_layout.argtypes = [ctypes.POINTER(Cfg), ctypes.c_int32, ctypes.POINTER(WsLayout)]
        L.moe_workspace_init.argtypes = [ctypes.POINTER(Cfg), ctypes.c_int32, _VP, ctypes.c_size_t, _VP]
        L.moe_route_select.argtypes = [ctypes.POINTER(Cfg), _VP, ctypes.c_int32, _VP, _VP, _VP, _VP, _VP,
                                       ctypes.c_size_t, _VP]
        L.moe_experts_decode.argtypes = [ctypes.POINTER(Cfg), _VP, ctypes.c_int32, _VP, ctypes.POINTER(Experts),
                                         _VP, _VP, ctypes.c_size_t, _VP]
        L.moe_experts_prefill.argtypes = [ctypes.POINTER(Cfg), _VP, ctypes.c_int32, _VP, ctypes.POINTER(Experts),
                                          _VP, _VP, ctypes.c_size_t, _VP]
        L.moe_layer_forward.argtypes = [ctypes.POINTER(Cfg), ctypes.POINTER(Layer), _VP, ctypes.c_int32, _VP, _VP,
                                        _VP, _VP, ctypes.c_size_t, _VP]
        L.moe_layer_forward_noalloc.argtypes = [ctypes.POINTER(Cfg), ctypes.POINTER(Layer), _VP, ctypes.c_int32,
                                                _VP, _VP, _VP, _VP]
        L.moe_stack_forward.argtypes = [ctypes.POINTER(Cfg), ctypes.POINTER(Layer), ctypes.c_int32, _VP,
                                         ctypes.c_int32, _VP, _VP, _VP, ctypes.c_size_t, _VP]
        L.moe_scores.argtypes = [_VP, ctypes.c_int64, ctypes.c_float, _VP, ctypes.c_int32, _VP]
        L.moe_scores_host.argtypes = [_VP, ctypes.c_int64, ctypes.c_float, _VP, ctypes.c_int32]
        L.moe_swiglu_host.argtypes = [_VP, _VP, ctypes.c_int64, ctypes.c_float, _VP]
        L.moe_time_next_launch.argtypes = [ctypes.c_int32, _VP, _VP]
        L.moe_read_probe.argtypes = [_VP, ctypes.c_uint64, _VP, ctypes.c_int32, _VP]
        L.moe_glibc_score_table.argtypes = [_VP, _VP, _VP, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
        L.moe_set_score_table.argtypes = [_VP, _VP, _VP, ctypes.c_int64]
        L.moe_cache_create.argtypes = [ctypes.POINTER(Cfg), ctypes.c_int32, ctypes.POINTER(_VP), ctypes.c_uint64,
                                       ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int32,
                                       ctypes.c_int32, ctypes.POINTER(_VP)]
        L.moe_cache_destroy.argtypes = [_VP]
        L.moe_cache_forward.argtypes = [_VP, ctypes.POINTER(Cfg), ctypes.POINTER(Layer), ctypes.c_int32, ctypes.c_int32,
                                        _VP, ctypes.c_int32, _VP, _VP, ctypes.c_int32, _VP, ctypes.c_size_t, _VP]
        L.moe_cache_prefetch.argtypes = [_VP, ctypes.c_int32, _VP, ctypes.c_int32, _VP]
        L.moe_cache_get_stats.argtypes = [_VP, ctypes.POINTER(CacheStats)]
        L.moe_cache_resident.argtypes = [_VP, ctypes.c_int32, _VP]
        L.moe_lru_simulate.argtypes = [ctypes.c_int32, ctypes.c_int64, _VP, _VP, ctypes.c_int32, _VP, _VP]
        L.moe_join_forward.argtypes = [_VP] * 6 + [ctypes.c_int64, _VP, _VP, _VP]
        L.moe_join_workspace_bytes.restype = ctypes.c_size_t
        L.moe_join_workspace_bytes.argtypes = [_VP, ctypes.c_int64]
        L.moe_join_backward.argtypes = [_VP] * 8 + [ctypes.c_int64] + [_VP] * 6 + [ctypes.c_size_t, _VP]
        for f in (L.moe_grouped_forward, L.moe_grouped_backward_x, L.moe_grouped_backward_w):
            f.argtypes = [_VP] * 4 + [ctypes.c_int64] + [_VP] * 3
        L.moe_adapter_workspace_bytes.restype = ctypes.c_size_t
        L.moe_adapter_workspace_bytes.argtypes = [_VP, ctypes.c_int64]
        L.moe_adapter_project.argtypes = [_VP] * 4 + [ctypes.c_int64, _VP, _VP, ctypes.c_size_t, _VP, _VP]
        L.moe_gated_forward.argtypes = [_VP] * 5 + [ctypes.c_int64] + [_VP] * 5
        L.moe_gated_backward_h.argtypes = [_VP] * 6 + [ctypes.c_int64] + [_VP] * 5
        L.moe_gated_backward_x.argtypes = [_VP] * 6 + [ctypes.c_int64] + [_VP] * 3
        L.moe_mx_quantise.argtypes = [_VP] * 2 + [ctypes.c_int64] + [_VP] * 3
        L.moe_mx_dequantise.argtypes = [_VP] * 3 + [ctypes.c_int64] + [_VP] * 2
        L.moe_mx_forward.argtypes = [_VP] * 6 + [ctypes.c_int64] + [_VP] * 3
        L.moe_mx_gated.argtypes = [_VP] * 8 + [ctypes.c_int64] + [_VP] * 3
        L.moe_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(code: int):
    if code != 0:
        raise MoeError(code, lib().moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        # the current device's current stream, without the Stream object that torch.cuda.current_stream() makes (3 us)
        import torch
        try:
            return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        except AttributeError:   # (a torch without that entry)
            return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def cfg_from_shape(shape) -> Cfg:
    return Cfg(shape.dim, shape.inter, shape.n_routed, shape.topk, int(shape.norm_topk_prob), shape.gate_temp,
               shape.route_scale, shape.swiglu_limit, int(shape.score_mode))


def header_words(cfg: Cfg) -> int:
    return int(lib().moe_header_words(ctypes.byref(cfg)))


def workspace_bytes(cfg: Cfg, max_m: int) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(cfg), max_m))


def workspace_layout(cfg: Cfg, max_m: int) -> dict:
    L = WsLayout()
    _check(lib().moe_workspace_layout(ctypes.byref(cfg), max_m, ctypes.byref(L)))
    return {n: getattr(L, n) for n, _ in WsLayout._fields_}


def workspace_init(cfg: Cfg, max_m: int, ws, stream=None):
    _check(lib().moe_workspace_init(ctypes.byref(cfg), max_m, _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)))


def route_select(cfg: Cfg, x, gate_w, bias, header, ws, logits=None, stream=None):
    m = x.shape[0]
    _check(lib().moe_route_select(ctypes.byref(cfg), _ptr(x), m, _ptr(gate_w), _ptr(bias), _ptr(logits),
                                  _ptr(header), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def experts_decode(cfg: Cfg, x, header, experts: Experts, y_routed, ws, stream=None):
    m = x.shape[0]
    _check(lib().moe_experts_decode(ctypes.byref(cfg), _ptr(x), m, _ptr(header), ctypes.byref(experts),
                                    _ptr(y_routed), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def experts_prefill(cfg: Cfg, x, header, experts: Experts, y_routed, ws, stream=None):
    m = x.shape[0]
    _check(lib().moe_experts_prefill(ctypes.byref(cfg), _ptr(x), m, _ptr(header), ctypes.byref(experts),
                                     _ptr(y_routed), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def layer_forward(cfg: Cfg, layer: Layer, x, out_bf16, ws, out_f32=None, header=None, stream=None):
    m = x.shape[0]
    _check(lib().moe_layer_forward(ctypes.byref(cfg), ctypes.byref(layer), _ptr(x), m, _ptr(out_bf16),
                                   _ptr(out_f32), _ptr(header), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)))


def layer_forward_noalloc(cfg: Cfg, layer: Layer, x, out_bf16, out_f32=None, header=None, stream=None):
    """The layer for m <= 8 tokens on the library's fixed scratch (no workspace argument)."""
    m = x.shape[0]
    _check(lib().moe_layer_forward_noalloc(ctypes.byref(cfg), ctypes.byref(layer), _ptr(x), m, _ptr(out_bf16),
                                           _ptr(out_f32), _ptr(header), _stream(stream)))


def stack_forward(cfg: Cfg, layers, xs, ws, out_f32=None, headers=None, stream=None):
    """xs: bf16 [n_layers+1, m, dim] (xs[0] the input); layers: a sequence of Layer."""
    n = len(layers)
    arr = (Layer * n)(*layers)
    m = xs.shape[1]
    _check(lib().moe_stack_forward(ctypes.byref(cfg), arr, n, _ptr(xs), m, _ptr(out_f32), _ptr(headers), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)))


def scores(logits, temp: float, out, flags: int = 0, stream=None):
    _check(lib().moe_scores(_ptr(logits), logits.numel(), ctypes.c_float(temp), _ptr(out), flags, _stream(stream)))


def scores_host(logits: np.ndarray, temp: float, flags: int = 0) -> np.ndarray:
    a = np.ascontiguousarray(logits, np.float32)
    out = np.empty_like(a)
    _check(lib().moe_scores_host(a.ctypes.data, a.size, ctypes.c_float(temp), out.ctypes.data, flags))
    return out


# flag bits of scores / scores_host
SCORES_EXTENDED = 1   # every exp/log1p through the extended-precision path
SCORES_GLIBC = 2      # the glibc mode's scores
SCORES_EXP_ONLY = 4   # the chain's exp step alone

MOE_SCORE_CR = 0
MOE_SCORE_GLIBC = 1
SCORE_INDEX_LEN = (1 << 24) + 1


def glibc_score_table():
    """(keys, vals, index) of the glibc score mode, as uint32 numpy arrays."""
    n = ctypes.c_int64(0)
    _check(lib().moe_glibc_score_table(None, None, None, 0, ctypes.byref(n)))
    keys = np.empty(n.value, np.uint32)
    vals = np.empty(n.value, np.uint32)
    index = np.empty(SCORE_INDEX_LEN, np.uint32)
    _check(lib().moe_glibc_score_table(keys.ctypes.data, vals.ctypes.data, index.ctypes.data, n.value,
                                       ctypes.byref(n)))
    return keys, vals, index


_score_tables = {}


def enable_glibc_scores(device=None):
    """Uploads the glibc score table to `device` (default: the current one) and
    registers it there; the tensors stay referenced here for the process."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    if dev.index in _score_tables:
        return
    keys, vals, index = glibc_score_table()
    with torch.cuda.device(dev):
        # (a host whose libm agrees everywhere still registers a non-NULL, empty table)
        t = [torch.from_numpy(a.view(np.int32) if a.size else np.zeros(1, np.int32)).to(dev)
             for a in (keys, vals, index)]
        torch.cuda.synchronize(dev)
        _check(lib().moe_set_score_table(t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr(), keys.size))
    _score_tables[dev.index] = t


def swiglu_host(g: np.ndarray, u: np.ndarray, limit: float) -> np.ndarray:
    g = np.ascontiguousarray(g, np.float32)
    u = np.ascontiguousarray(u, np.float32)
    out = np.empty_like(g)
    _check(lib().moe_swiglu_host(g.ctypes.data, u.ctypes.data, g.size, ctypes.c_float(limit), out.ctypes.data))
    return out


def time_next_launch(which: int, ev_begin, ev_end):
    """Bracket the next launch of kernel `which` with two torch.cuda.Event objects."""
    b = None if ev_begin is None else ctypes.c_void_p(ev_begin.cuda_event)
    e = None if ev_end is None else ctypes.c_void_p(ev_end.cuda_event)
    _check(lib().moe_time_next_launch(which, b, e))


def read_probe(buf, nbytes: int, sink, blocks: int, stream=None):
    """Stream `nbytes` of the device tensor `buf` through the library's read-only probe kernel."""
    _check(lib().moe_read_probe(_ptr(buf), nbytes, _ptr(sink), blocks, _stream(stream)))


class ExpertCache:
    """An expert cache (moe_cache_*): n_slots device slots over the host-resident
    experts of len(host_arenas) layers (host tensors or addresses)."""

    def __init__(self, cfg: Cfg, host_arenas, stride: int, gate_off: int, up_off: int, down_off: int, n_slots: int,
                 max_m: int):
        ptrs = [a if isinstance(a, int) else a.data_ptr() for a in host_arenas]
        arr = (_VP * len(ptrs))(*ptrs)
        h = _VP()
        _check(lib().moe_cache_create(ctypes.byref(cfg), len(ptrs), arr, stride, gate_off, up_off, down_off, n_slots,
                                      max_m, ctypes.byref(h)))
        self.h, self.cfg = h, cfg

    def forward(self, layers, xs, ws, first_layer: int = 0, out_f32=None, headers=None, prefetch_k: int = 0,
                stream=None):
        """xs: bf16 [n_layers+1, m, dim] (xs[0] the input); layers: the cache's layers first_layer.. (Layer)."""
        n = len(layers)
        arr = (Layer * n)(*layers)
        _check(lib().moe_cache_forward(self.h, ctypes.byref(self.cfg), arr, first_layer, n, _ptr(xs), xs.shape[1],
                                       _ptr(out_f32), _ptr(headers), prefetch_k, _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream)))

    def prefetch(self, layer: int, experts, stream=None):
        a = np.ascontiguousarray(experts, np.int32)
        _check(lib().moe_cache_prefetch(self.h, layer, a.ctypes.data, a.size, _stream(stream)))

    def stats(self) -> dict:
        st = CacheStats()
        _check(lib().moe_cache_get_stats(self.h, ctypes.byref(st)))
        return {n: getattr(st, n) for n, _ in CacheStats._fields_}

    def resident(self, layer: int) -> np.ndarray:
        out = np.empty(self.cfg.n_routed, np.int32)
        _check(lib().moe_cache_resident(self.h, layer, out.ctypes.data))
        return out

    def close(self):
        if self.h:
            lib().moe_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def lru_simulate(n_slots: int, n_keys: int, batches):
    """The cache's slot assignment on the host: each batch a list of keys; returns (slots, misses) per request."""
    keys = np.ascontiguousarray(np.concatenate([np.asarray(b, np.int64) for b in batches]) if batches else
                                np.zeros(0, np.int64))
    lens = np.ascontiguousarray([len(b) for b in batches], np.int32)
    slots = np.empty(keys.size, np.int32)
    miss = np.empty(keys.size, np.int32)
    _check(lib().moe_lru_simulate(n_slots, n_keys, keys.ctypes.data, lens.ctypes.data, len(batches),
                                  slots.ctypes.data, miss.ctypes.data))
    return slots, miss


# ---- operators beside the layer -------------------------------------------
MOE_TYPE_BF16, MOE_TYPE_FP16, MOE_TYPE_F32 = 0, 1, 2
MOE_STATUS_BAD_OFFSETS = 8
MOE_STATUS_BAD_ADAPTER = 16
MOE_JOIN_MAX_DIM = 16384
MOE_GROUPED_MAX_GROUPS = 1024
MOE_GROUPED_MAX_STRIDE = 1 << 22
MOE_GROUPED_MAX_ROWS = 0x7fffff00
MOE_ACT_SILU, MOE_ACT_GELU = 0, 1
MOE_MX_FLOOR, MOE_MX_CEIL = 0, 1
MOE_MX_MAX_K = 1 << 22
MOE_MX_MAX_ROWS = 0x7fffffff
MOE_ADAPTER_MAX_ADAPTERS = 1024
MOE_ADAPTER_MAX_RANK = 1024
MOE_ADAPTER_MAX_TOKENS = 1 << 20


def type_code(dtype) -> int:
    """The MOE_TYPE_* code of a torch dtype (a code passes through)."""
    if isinstance(dtype, int):
        return dtype
    code = {"torch.bfloat16": MOE_TYPE_BF16, "torch.float16": MOE_TYPE_FP16, "torch.float32": MOE_TYPE_F32}.get(
        str(dtype))
    if code is None:
        raise MoeError(-1, f"element type must be bfloat16, float16 or float32 (got {dtype})")
    return code


def _addr(t):
    return None if t is None else t.data_ptr()


_native = None


def _tensors():
    """The native module that holds these calls' tensors against their description and makes the calls
    (csrc/moe_tensors.cpp)."""
    global _native
    if _native is None:
        L = lib()
        import torch  # noqa: F401  (its libraries are the module's)
        try:
            from . import _tensors as native
        except ImportError as e:
            raise ImportError(f"{TENSORS_PATH} is not built: run __graft_entry__.build()") from e
        native.bind(MoeError, *(ctypes.cast(f, _VP).value for f in (
            L.moe_join_forward, L.moe_join_backward, L.moe_grouped_forward, L.moe_grouped_backward_x,
            L.moe_grouped_backward_w, L.moe_adapter_project, L.moe_gated_forward, L.moe_gated_backward_h,
            L.moe_gated_backward_x, L.moe_mx_quantise, L.moe_mx_dequantise, L.moe_mx_forward, L.moe_mx_gated,
            L.moe_last_error)))
        _native = native
    return _native


class Join(ctypes.Structure):
    """moe_join: how a block joins a residual stream (norms after and before, gate, residual scale).
    Strides default to contiguous rows of dim."""
    _fields_ = [("dim", ctypes.c_int32), ("type", ctypes.c_int32), ("residual_type", ctypes.c_int32),
                ("gate_rows", ctypes.c_int32), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("x_out_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64)]

    def __init__(self, dim: int, dtype, residual=None, gate_rows: bool = False, scale: float = 1.0, eps: float = 1e-6,
                 x_stride: int | None = None, x_out_stride: int | None = None, b_stride: int | None = None,
                 gate_stride: int | None = None, y_stride: int | None = None):
        t = type_code(dtype)
        super().__init__(dim, t, t if residual is None else type_code(residual), int(gate_rows), scale, eps,
                         *(dim if v is None else v for v in (x_stride, x_out_stride, b_stride, gate_stride, y_stride)))


def join_forward(j: Join, x, block, w_post, gate, w_pre, x_out, y, stream=None):
    """x_out = x + scale * gate * norm(block, w_post), y = norm(x_out, w_pre); block, w_post, gate, w_pre with y,
    and (without a block) x_out may be None."""
    _tensors().join_forward(j, x, block, w_post, gate, w_pre, x_out, y, _stream(stream))


def join_workspace_bytes(j: Join, max_m: int) -> int:
    return int(lib().moe_join_workspace_bytes(ctypes.byref(j), max_m))


def join_backward(j: Join, dy, dx_out, x_out, block, w_post, gate, w_pre, dx, dblock, dw_post, dgate, dw_pre, ws,
                  stream=None):
    """The gradients of join_forward: dx, dblock, dw_post, dgate, dw_pre (None where not wanted)."""
    _tensors().join_backward(j, dy, dx_out, x_out, block, w_post, gate, w_pre, dx, dblock, dw_post, dgate, dw_pre, ws,
                             _stream(stream))


class Grouped(ctypes.Structure):
    """moe_grouped: products of rows sorted by group with one n x k weight per group.
    Strides default to contiguous rows and weights."""
    _fields_ = [("n_groups", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("type", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("w_stride", ctypes.c_int64), ("w_group_stride", ctypes.c_int64)]

    def __init__(self, n_groups: int, n: int, k: int, dtype, out=None, x_stride: int | None = None,
                 y_stride: int | None = None, w_stride: int | None = None, w_group_stride: int | None = None):
        t = type_code(dtype)
        ws = k if w_stride is None else w_stride
        super().__init__(n_groups, n, k, t, t if out is None else type_code(out), k if x_stride is None else x_stride,
                         n if y_stride is None else y_stride, ws, n * ws if w_group_stride is None else w_group_stride)


def grouped_forward(g: Grouped, x, w, offsets, y, status=None, stream=None):
    """y[r] = w[group of r] @ x[r]; offsets: int32 [n_groups + 1] on the device."""
    _tensors().grouped_forward(g, x, w, offsets, y, status, _stream(stream))


def grouped_backward_x(g: Grouped, dy, w, offsets, dx, status=None, stream=None):
    """dx[r] = w[group of r]^T @ dy[r]."""
    _tensors().grouped_backward_x(g, dy, w, offsets, dx, status, _stream(stream))


def grouped_backward_w(g: Grouped, dy, x, offsets, dw, status=None, stream=None):
    """dw[g] = the sum of dy[r] x[r]^T over the group's rows."""
    _tensors().grouped_backward_w(g, dy, x, offsets, dw, status, _stream(stream))


def act_code(act) -> int:
    """The MOE_ACT_* code of "silu" or "gelu" (a code passes through)."""
    if isinstance(act, int):
        return act
    code = {"silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}.get(act)
    if code is None:
        raise MoeError(-1, f"act must be silu or gelu (got {act!r})")
    return code


class Gated(ctypes.Structure):
    """moe_gated: a gated feed-forward block per group of rows, act(min(g, limit)) * clamp(u, -limit, limit) between
    its projections (limit 0 or None: no clamps). dx: the type of the input's gradient. Strides default to contiguous
    rows and weights."""
    _fields_ = [("n_groups", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("type", ctypes.c_int32),
                ("dx_type", ctypes.c_int32), ("act", ctypes.c_int32), ("limit", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("h_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("w_stride", ctypes.c_int64), ("w_group_stride", ctypes.c_int64),
                ("down_stride", ctypes.c_int64), ("down_group_stride", ctypes.c_int64)]

    def __init__(self, n_groups: int, n: int, k: int, dtype, act="silu", limit: float | None = None, dx=None,
                 x_stride: int | None = None, h_stride: int | None = None, gate_stride: int | None = None,
                 y_stride: int | None = None, w_stride: int | None = None, w_group_stride: int | None = None,
                 down_stride: int | None = None, down_group_stride: int | None = None):
        t = type_code(dtype)
        ws = k if w_stride is None else w_stride
        ds = n if down_stride is None else down_stride
        super().__init__(n_groups, n, k, t, t if dx is None else type_code(dx), act_code(act), limit or 0.0,
                         k if x_stride is None else x_stride, n if h_stride is None else h_stride,
                         n if gate_stride is None else gate_stride, k if y_stride is None else y_stride, ws,
                         n * ws if w_group_stride is None else w_group_stride, ds,
                         k * ds if down_group_stride is None else down_group_stride)


def gated_forward(g: Gated, x, w_gate, w_up, offsets, h, gate=None, up=None, status=None, stream=None):
    """h[r] = act(w_gate[group of r] @ x[r]) * (w_up[group of r] @ x[r]); gate and up: the two products, kept for the
    gradients."""
    _tensors().gated_forward(g, x, w_gate, w_up, offsets, h, gate, up, status, _stream(stream))


def gated_backward_h(g: Gated, dy, w_down, gate, up, offsets, dgate, dup, h=None, status=None, stream=None):
    """dgate and dup of the kept gate and up, for h's gradient w_down[group of r]^T @ dy[r]; h: made again."""
    _tensors().gated_backward_h(g, dy, w_down, gate, up, offsets, dgate, dup, h, status, _stream(stream))


def gated_backward_x(g: Gated, dgate, dup, w_gate, w_up, offsets, dx, status=None, stream=None):
    """dx[r] = w_gate[group of r]^T @ dgate[r] + w_up[group of r]^T @ dup[r]."""
    _tensors().gated_backward_x(g, dgate, dup, w_gate, w_up, offsets, dx, status, _stream(stream))


class MxRows(ctypes.Structure):
    """moe_mx_rows: rows of k elements of dtype and their microscaled 4-bit form, codes [rows, (k + 1) // 2] and scales
    [rows, (k + 31) // 32] bytes. scale "floor" or "ceil": which power of two the largest of 32 elements gives. Strides
    (of x in elements, of the others in bytes) default to contiguous rows."""
    _fields_ = [("k", ctypes.c_int32), ("type", ctypes.c_int32), ("scale", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("code_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64)]

    def __init__(self, k: int, dtype, scale="floor", x_stride: int | None = None, code_stride: int | None = None,
                 scale_stride: int | None = None):
        rule = scale if isinstance(scale, int) else {"floor": MOE_MX_FLOOR, "ceil": MOE_MX_CEIL}.get(scale)
        if rule is None:
            raise MoeError(-1, f"scale must be floor or ceil (got {scale!r})")
        super().__init__(k, type_code(dtype), rule, k if x_stride is None else x_stride,
                         (k + 1) // 2 if code_stride is None else code_stride,
                         (k + 31) // 32 if scale_stride is None else scale_stride)


def mx_quantise(p: MxRows, x, codes, scales, stream=None):
    """Rows of x to 4-bit codes and the scales of 32 elements each."""
    _tensors().mx_quantise(p, x, codes, scales, _stream(stream))


def mx_dequantise(p: MxRows, codes, scales, x, stream=None):
    """The values that codes and scales stand for, rounded to x's type."""
    _tensors().mx_dequantise(p, codes, scales, x, _stream(stream))


class Mx(ctypes.Structure):
    """moe_mx: products grouped by expert of rows and weights in microscaled 4-bit floats, out: the outputs' type; act and
    limit: as Gated, for mx_gated. Strides (of the outputs in elements, of the others in bytes) default to contiguous rows
    and weights."""
    _fields_ = [("n_groups", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("out_type", ctypes.c_int32),
                ("act", ctypes.c_int32), ("limit", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("x_scale_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("w_stride", ctypes.c_int64),
                ("w_group_stride", ctypes.c_int64), ("w_scale_stride", ctypes.c_int64),
                ("w_scale_group_stride", ctypes.c_int64)]

    def __init__(self, n_groups: int, n: int, k: int, out, act="silu", limit: float | None = None,
                 x_stride: int | None = None, x_scale_stride: int | None = None, y_stride: int | None = None,
                 w_stride: int | None = None, w_group_stride: int | None = None, w_scale_stride: int | None = None,
                 w_scale_group_stride: int | None = None):
        codes, blocks = (k + 1) // 2, (k + 31) // 32
        ws, ss = codes if w_stride is None else w_stride, blocks if w_scale_stride is None else w_scale_stride
        super().__init__(n_groups, n, k, type_code(out), act_code(act), limit or 0.0, codes if x_stride is None else x_stride,
                         blocks if x_scale_stride is None else x_scale_stride, n if y_stride is None else y_stride, ws,
                         n * ws if w_group_stride is None else w_group_stride, ss,
                         n * ss if w_scale_group_stride is None else w_scale_group_stride)


def mx_forward(m: Mx, x, x_scale, w, w_scale, offsets, y, status=None, stream=None):
    """y[r] = w[group of r] @ x[r] of codes and scales (as mx_quantise makes them)."""
    _tensors().mx_forward(m, x, x_scale, w, w_scale, offsets, y, status, _stream(stream))


def mx_gated(m: Mx, x, x_scale, w_gate, w_gate_scale, w_up, w_up_scale, offsets, h, status=None, stream=None):
    """h[r] = act(w_gate[group of r] @ x[r]) * (w_up[group of r] @ x[r]) of codes and scales."""
    _tensors().mx_gated(m, x, x_scale, w_gate, w_gate_scale, w_up, w_up_scale, offsets, h, status, _stream(stream))


class Adapters(ctypes.Structure):
    """moe_adapters: the low-rank adapters a [n_adapters, rank, k] and b [n_adapters, n, rank] (device tensors, kept
    here) beside a shared n x k projection; factor f32 [n_adapters] or None. Strides default to contiguous rows."""
    _fields_ = [("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("a", _VP), ("b", _VP), ("factor", _VP),
                ("x_stride", ctypes.c_int64), ("w_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("a_stride", ctypes.c_int64), ("a_group_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("b_group_stride", ctypes.c_int64)]

    def __init__(self, a, b, factor=None, out=None, x_stride: int | None = None, w_stride: int | None = None,
                 out_stride: int | None = None):
        count, rank, k = a.shape
        n = b.shape[1]
        if tuple(b.shape) != (count, n, rank) or a.dtype != b.dtype:
            raise MoeError(-1, f"adapters: a {tuple(a.shape)} {a.dtype} and b {tuple(b.shape)} {b.dtype} do not fit")
        if (k > 1 and a.stride(2) != 1) or (rank > 1 and b.stride(2) != 1):
            raise MoeError(-1, "adapters: the rows of a and b must be contiguous")
        if factor is not None and (type_code(factor.dtype) != MOE_TYPE_F32 or tuple(factor.shape) != (count,) or
                                   not factor.is_contiguous()):
            raise MoeError(-1, "adapters: factor must be contiguous f32 [n_adapters]")
        t = type_code(a.dtype)
        super().__init__(count, rank, n, k, t, t if out is None else type_code(out), _addr(a), _addr(b), _addr(factor),
                         k if x_stride is None else x_stride, k if w_stride is None else w_stride,
                         n if out_stride is None else out_stride, a.stride(1), a.stride(0), b.stride(1), b.stride(0))
        self._kept = (a, b, factor)


def adapter_workspace_bytes(p: Adapters, max_m: int) -> int:
    return int(lib().moe_adapter_workspace_bytes(ctypes.byref(p), max_m))


def adapter_project(p: Adapters, x, w, index, out, ws, status=None, stream=None):
    """out[t] = w @ x[t] + factor[a] * b[a] @ (a[a] @ x[t]) with a = index[t] (-1: w @ x[t] alone)."""
    _tensors().adapter_project(p, x, w, index, out, ws, status, _stream(stream))
