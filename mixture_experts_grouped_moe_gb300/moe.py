"""Thin ctypes binding of libmoe_gb300 (include/moe.h), same names as the C ABI.

Only argument marshalling lives here: tensors become raw pointers, the
current torch CUDA stream becomes the `stream` argument, and a negative
status raises MoEError.  Every step of the layer runs in the CUDA library;
there is no Python or CPU fallback.  If the library is missing the first
call raises (build it with `mixture_experts_grouped_moe_gb300.build`).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

from . import build as _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_TIMEOUT = -5

MOE_BF16 = 0
MOE_FP8_BLOCK128 = 1
MOE_FP8_TOKEN = 2
MOE_MXFP4 = 3
MOE_MODE_GROUPED = 0
MOE_MODE_SWAP = 1

MOE_ROW_BF16 = 0
MOE_ROW_FP16 = 1
MOE_ROW_FP32 = 2
MOE_GATE_NONE = 0
MOE_GATE_CHANNEL = 1
MOE_GATE_TOKEN = 2
MOE_GATE_FULL = 3
MOE_GEMM_BLOCK_WS_BYTES = 64

EXPORTED = [
    "moe_status_string", "moe_version", "moe_align_sort_sizes", "moe_block_size_m_heuristic",
    "moe_ksplit_heuristic", "moe_plan", "moe_fused_workspace_size", "moe_workspace_layout",
    "moe_workspace_status", "moe_route_topk", "moe_align_sort_workspace_size", "moe_align_sort",
    "moe_quantize_fp8_act", "moe_quantize_fp8_weights", "moe_quantize_fp8_rows", "moe_fused_forward",
    "moe_host_staging_bytes", "moe_fused_forward_host", "moe_align_sort_noalloc", "moe_quantize_mxfp4",
    "moe_train_workspace_size", "moe_fused_forward_train", "moe_fused_backward", "moe_options_init",
    "moe_fused_forward_ex", "moe_align_sort_map", "moe_align_sort_drop", "moe_permute",
    "moe_permute_fp8", "moe_permute_backward",
    "moe_unpermute", "moe_unpermute_backward", "moe_gemm_fp8_block", "moe_wgrad_fp8_block",
    "moe_quantize_fp8_act_t", "moe_block_norm", "moe_block_norm_workspace_size", "moe_block_norm_backward",
]


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


class moe_plan_t(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("block_m", ctypes.c_int), ("split_k1", ctypes.c_int),
                ("split_k2", ctypes.c_int), ("max_padded", ctypes.c_int64), ("max_blocks", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_size_t)]


class moe_options_t(ctypes.Structure):
    _fields_ = [("gemm_pair", ctypes.c_int), ("one_stage", ctypes.c_int), ("pdl_mask", ctypes.c_int),
                ("stage_events", ctypes.c_void_p), ("h_wait_limit_us", ctypes.c_uint),
                ("unsatisfiable_h_wait", ctypes.c_int), ("light_tiles", ctypes.c_int), ("tc_router", ctypes.c_int)]


class moe_ws_layout_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "status", "topk_ids", "topk_weights", "sorted_ids", "sorted_weights", "sorted_expert_ids",
        "num_tokens_post_padded", "expert_counts", "x_sorted", "x_scales", "inter", "inter_scales", "inter_h",
        "y", "router_logits", "total")]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_build.LIB):
            if not build_if_missing:
                raise RuntimeError(f"CUDA library not built: {_build.LIB} is missing "
                                   "(run mixture_experts_grouped_moe_gb300.build.build())")
            _build.build()
        lib = ctypes.CDLL(_build.LIB)
        P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        sig = {
            "moe_status_string": (ctypes.c_char_p, [I]),
            "moe_version": (I, []),
            "moe_align_sort_sizes": (I, [I, I, I, I, P, P]),
            "moe_block_size_m_heuristic": (I, [I, I, I, I, I, P, I]),
            "moe_ksplit_heuristic": (I, [I, I, I, I, I, I, I]),
            "moe_plan": (I, [I, I, I, I, I, I, I, I, I, P]),
            "moe_fused_workspace_size": (SZ, [I, I, I, I, I, I, I, I]),
            "moe_workspace_layout": (I, [I, I, I, I, I, I, I, I, P]),
            "moe_workspace_status": (I, [P, P, P]),
            "moe_route_topk": (I, [P, P, P, I, I, I, I, I, P, P, P, P]),
            "moe_align_sort_workspace_size": (SZ, [I, I, I]),
            "moe_align_sort": (I, [P, P, I, I, I, I, P, P, P, P, P, P, SZ, P]),
            "moe_quantize_fp8_act": (I, [P, I64, I, P, P, P]),
            "moe_quantize_fp8_weights": (I, [P, I64, I, P, P, P]),
            "moe_quantize_fp8_rows": (I, [P, I64, I, P, P, P]),
            "moe_fused_forward": (I, [I, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, SZ, P]),
            "moe_host_staging_bytes": (SZ, [I, I]),
            "moe_fused_forward_host": (I, [I, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, SZ, P]),
            "moe_options_init": (I, [P]),
            "moe_fused_forward_ex": (I, [I, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, SZ, P, P]),
            "moe_train_workspace_size": (SZ, [I, I, I, I, I]),
            "moe_fused_forward_train": (I, [P, P, P, P, P, I, I, I, I, I, P, P, SZ, P, P]),
            "moe_fused_backward": (I, [P, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, SZ, P, P]),
            "moe_quantize_mxfp4": (I, [P, I64, I, P, P, I, P]),
            "moe_align_sort_noalloc": (I, [P, P, I, I, I, I, P, P, P, P, P, P]),
            "moe_align_sort_map": (I, [P, P, I, I, I, I, P, P, P, P, P, P, P, SZ, P]),
            "moe_align_sort_drop": (I, [P, P, I, I, I, I, P, P, P, P, P, P, P, P, SZ, P]),
            "moe_permute": (I, [I, P, I64, P, P, P, I, I, I, I64, I, P, P]),
            "moe_permute_fp8": (I, [P, I64, P, P, P, I, I, I, I64, I, P, P, P]),
            "moe_permute_backward": (I, [I, P, P, I, I, I, I64, P, I64, P]),
            "moe_unpermute": (I, [I, P, P, P, I, I, I, I64, P, I64, P]),
            "moe_unpermute_backward": (I, [I, P, I64, P, P, P, P, P, I, I, I, I64, I, P, P, P]),
            "moe_gemm_fp8_block": (I, [P, P, I, P, P, I64, I, I, I, I, P, P, I, P, I64, P, SZ, P]),
            "moe_wgrad_fp8_block": (I, [P, P, P, P, I64, I, I, I, P, P, I, P, SZ, P]),
            "moe_quantize_fp8_act_t": (I, [P, I64, I64, I, P, I, I, P, P, I64, P, P]),
            "moe_block_norm": (I, [I, P, P, P, I, P, P, I64, I, F, F, F, P, P, P, P, P]),
            "moe_block_norm_workspace_size": (SZ, [I64, I]),
            "moe_block_norm_backward": (I, [I, P, P, P, I, P, P, P, P, P, P, I64, I, F, F, P, P, P, P, P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
        return lib


def _p(t):
    """Raw pointer of a tensor / int / None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _pn(t, n, instead=256):
    """Raw pointer of a tensor of n rows.  An empty tensor's is null, which the entry points turn down where
    they need a pointer; with n = 0 they touch nothing behind it, so any aligned address (`instead`) will do."""
    if n:
        return t if t is None or isinstance(t, int) else t.data_ptr()
    return _p(t) or (_p(instead) if t is not None else None)


_raw_stream = None  # () -> cudaStream_t of the current device's current stream


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    global _raw_stream
    if _raw_stream is None:
        import torch
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if get is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            # without building a Stream object: 3.0 -> 0.4 us of every call's host time
            _raw_stream = lambda: get(torch.cuda.current_device())  # noqa: E731
    return _raw_stream()


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoEError(fn, rc)
    return rc


def status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def moe_version() -> int:
    return load().moe_version()


def moe_align_sort_sizes(T, k, E, block_m):
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check("moe_align_sort_sizes", load().moe_align_sort_sizes(T, k, E, block_m, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def moe_block_size_m_heuristic(token, topk, expert, inter_dim, units, candidates=(32, 64, 128)):
    arr = (ctypes.c_int * len(candidates))(*candidates)
    r = load().moe_block_size_m_heuristic(token, topk, expert, inter_dim, units, arr, len(candidates))
    if r < 0:
        raise MoEError("moe_block_size_m_heuristic", r)
    return r


def moe_ksplit_heuristic(token, topk, expert, inter_dim, model_dim, units, block_m):
    r = load().moe_ksplit_heuristic(token, topk, expert, inter_dim, model_dim, units, block_m)
    if r < 0:
        raise MoEError("moe_ksplit_heuristic", r)
    return r


def moe_plan(dtype, T, H, I, E, k, block_m=0, split_k=0, num_sms=0) -> moe_plan_t:
    p = moe_plan_t()
    _check("moe_plan", load().moe_plan(dtype, T, H, I, E, k, block_m, split_k, num_sms, ctypes.byref(p)))
    return p


def moe_fused_workspace_size(dtype, T, H, I, E, k, block_m=0, split_k=0) -> int:
    return load().moe_fused_workspace_size(dtype, T, H, I, E, k, block_m, split_k)


def moe_workspace_layout(dtype, T, H, I, E, k, block_m=0, split_k=0) -> moe_ws_layout_t:
    lay = moe_ws_layout_t()
    _check("moe_workspace_layout",
           load().moe_workspace_layout(dtype, T, H, I, E, k, block_m, split_k, ctypes.byref(lay)))
    return lay


def moe_workspace_status(ws, stream=None) -> int:
    v = ctypes.c_int()
    _check("moe_workspace_status", load().moe_workspace_status(_p(ws), ctypes.byref(v), _stream(stream)))
    return v.value


def moe_route_topk(x, W_router, bias, T, H, E, k, topk_ids, topk_weights, logits=None, stream=None,
                   renormalize=True):
    return _check("moe_route_topk", load().moe_route_topk(
        _p(x), _p(W_router), _p(bias), T, H, E, k, 1 if renormalize else 0, _p(topk_ids), _p(topk_weights),
        _p(logits), _stream(stream)))


def moe_align_sort_workspace_size(T, k, E) -> int:
    return load().moe_align_sort_workspace_size(T, k, E)


def moe_align_sort(topk_ids, topk_weights, T, k, E, block_m, sorted_ids, sorted_weights, sorted_expert_ids,
                   num_tokens_post_padded, expert_counts, ws, ws_bytes, stream=None):
    return _check("moe_align_sort", load().moe_align_sort(
        _p(topk_ids), _p(topk_weights), T, k, E, block_m, _p(sorted_ids), _p(sorted_weights),
        _p(sorted_expert_ids), _p(num_tokens_post_padded), _p(expert_counts), _p(ws), ws_bytes,
        _stream(stream)))


def moe_align_sort_noalloc(topk_ids, topk_weights, T, k, E, block_m, sorted_ids, sorted_weights,
                           sorted_expert_ids, num_tokens_post_padded, expert_counts, stream=None):
    """moe_align_sort with the library's fixed device scratch instead of a caller workspace."""
    return _check("moe_align_sort_noalloc", load().moe_align_sort_noalloc(
        _p(topk_ids), _p(topk_weights), T, k, E, block_m, _p(sorted_ids), _p(sorted_weights),
        _p(sorted_expert_ids), _p(num_tokens_post_padded), _p(expert_counts), _stream(stream)))


def moe_quantize_fp8_act(X, R, C, q, s, stream=None):
    return _check("moe_quantize_fp8_act", load().moe_quantize_fp8_act(_p(X), R, C, _p(q), _p(s), _stream(stream)))


def moe_quantize_fp8_weights(W, R, C, q, s, stream=None):
    return _check("moe_quantize_fp8_weights",
                  load().moe_quantize_fp8_weights(_p(W), R, C, _p(q), _p(s), _stream(stream)))


def moe_quantize_fp8_rows(X, R, C, q, s, stream=None):
    return _check("moe_quantize_fp8_rows", load().moe_quantize_fp8_rows(_p(X), R, C, _p(q), _p(s), _stream(stream)))


def moe_quantize_mxfp4(X, R, C, q, s, tiled=False, stream=None):
    return _check("moe_quantize_mxfp4",
                  load().moe_quantize_mxfp4(_p(X), R, C, _p(q), _p(s), 1 if tiled else 0, _stream(stream)))


def moe_fused_forward(dtype, x, W_router, router_bias, W_gate_up, w1_scale, W_down, w2_scale, T, H, I, E, k,
                      block_m, split_k, out, ws, ws_bytes, stream=None):
    return _check("moe_fused_forward", load().moe_fused_forward(
        dtype, _p(x), _p(W_router), _p(router_bias), _p(W_gate_up), _p(w1_scale), _p(W_down), _p(w2_scale),
        T, H, I, E, k, block_m, split_k, _p(out), _p(ws), ws_bytes, _stream(stream)))


def moe_host_staging_bytes(T, H) -> int:
    return load().moe_host_staging_bytes(T, H)


def moe_fused_forward_host(dtype, x_host, W_router, router_bias, W_gate_up, w1_scale, W_down, w2_scale, T, H, I,
                           E, k, block_m, split_k, out_host, ws, ws_bytes, stream=None):
    return _check("moe_fused_forward_host", load().moe_fused_forward_host(
        dtype, _p(x_host), _p(W_router), _p(router_bias), _p(W_gate_up), _p(w1_scale), _p(W_down), _p(w2_scale),
        T, H, I, E, k, block_m, split_k, _p(out_host), _p(ws), ws_bytes, _stream(stream)))


class Options:
    """Per-call choices of moe_fused_forward_ex (see moe_options_t in include/moe.h).

    Keyword arguments override the library's defaults: gemm_pair (-1/0/1), one_stage (0/1),
    pdl_mask (-1 or a mask), stage_events (7 torch.cuda.Event or None), h_wait_limit_us,
    unsatisfiable_h_wait (0/1, for the timeout test only), light_tiles (-1/0/1), tc_router (-1/0/1)."""

    def __init__(self, **kw):
        self.c = moe_options_t()
        _check("moe_options_init", load().moe_options_init(ctypes.byref(self.c)))
        self._events = None
        for key, val in kw.items():
            setattr(self, key, val)

    def __setattr__(self, key, val):
        if key in ("c", "_events"):
            object.__setattr__(self, key, val)
        elif key == "stage_events":
            if val is None:
                self._events = None
                self.c.stage_events = None
            else:
                arr = (ctypes.c_void_p * len(val))(*[e.cuda_event for e in val])
                self._events = (arr, list(val))  # keep both alive while the options are in use
                self.c.stage_events = ctypes.cast(arr, ctypes.c_void_p)
        elif key in dict(moe_options_t._fields_):
            setattr(self.c, key, val)
        else:
            raise AttributeError(key)

    def __getattr__(self, key):
        if key in dict(moe_options_t._fields_):
            return getattr(self.c, key)
        raise AttributeError(key)


def _opt(options):
    if options is None:
        return None
    return ctypes.byref(options.c if isinstance(options, Options) else options)


def moe_fused_forward_ex(dtype, x, W_router, router_bias, W_gate_up, w1_scale, W_down, w2_scale, T, H, I, E, k,
                         block_m, split_k, out, ws, ws_bytes, options=None, stream=None):
    return _check("moe_fused_forward_ex", load().moe_fused_forward_ex(
        dtype, _p(x), _p(W_router), _p(router_bias), _p(W_gate_up), _p(w1_scale), _p(W_down), _p(w2_scale),
        T, H, I, E, k, block_m, split_k, _p(out), _p(ws), ws_bytes, _opt(options), _stream(stream)))


def moe_train_workspace_size(T, H, I, E, k) -> int:
    return load().moe_train_workspace_size(T, H, I, E, k)


def moe_fused_forward_train(x, W_router, router_bias, W_gate_up, W_down, T, H, I, E, k, out, ws, ws_bytes,
                            options=None, stream=None):
    return _check("moe_fused_forward_train", load().moe_fused_forward_train(
        _p(x), _p(W_router), _p(router_bias), _p(W_gate_up), _p(W_down), T, H, I, E, k, _p(out), _p(ws), ws_bytes,
        _opt(options), _stream(stream)))


def moe_fused_backward(x, W_router, router_bias, W_gate_up, W_down, dout, T, H, I, E, k, dx, dW_gate_up, dW_down,
                       dW_router, dbias, ws, ws_bytes, options=None, stream=None):
    return _check("moe_fused_backward", load().moe_fused_backward(
        _p(x), _p(W_router), _p(router_bias), _p(W_gate_up), _p(W_down), _p(dout), T, H, I, E, k, _p(dx),
        _p(dW_gate_up), _p(dW_down), _p(dW_router), _p(dbias), _p(ws), ws_bytes, _opt(options), _stream(stream)))


# ------------------------------------------------- operators around the layer

def moe_align_sort_map(topk_ids, topk_weights, T, k, E, block_m, sorted_ids, sorted_weights, sorted_expert_ids,
                       num_tokens_post_padded, expert_counts, slot_pos, ws, ws_bytes, stream=None):
    """moe_align_sort that also writes slot_pos, the sorted position of each slot."""
    P = T * k + E * block_m - k
    return _check("moe_align_sort_map", load().moe_align_sort_map(
        _pn(topk_ids, T), _pn(topk_weights, T), T, k, E, block_m, _pn(sorted_ids, P), _pn(sorted_weights, P),
        _pn(sorted_expert_ids, P), _p(num_tokens_post_padded), _p(expert_counts), _pn(slot_pos, T), _p(ws), ws_bytes,
        _stream(stream)))


def moe_align_sort_drop(topk_ids, topk_weights, T, k, E, block_m, sorted_ids, sorted_weights, sorted_expert_ids,
                        num_tokens_post_padded, expert_counts, slot_pos, num_left_out, ws, ws_bytes, stream=None):
    """moe_align_sort_map where an id outside [0, E) leaves its slot out instead of refusing the routing."""
    P = T * k + E * block_m - k
    return _check("moe_align_sort_drop", load().moe_align_sort_drop(
        _pn(topk_ids, T), _pn(topk_weights, T), T, k, E, block_m, _pn(sorted_ids, P), _pn(sorted_weights, P),
        _pn(sorted_expert_ids, P), _p(num_tokens_post_padded), _p(expert_counts), _pn(slot_pos, T), _p(num_left_out),
        _p(ws), ws_bytes, _stream(stream)))


def moe_permute(row_type, x, ld_x, slot_pos, sorted_ids, num_tokens_post_padded, T, k, H, P, zero_padding, xs,
                stream=None):
    return _check("moe_permute", load().moe_permute(
        row_type, _pn(x, T), ld_x, _pn(slot_pos, T), _pn(sorted_ids, T and P), _p(num_tokens_post_padded), T, k, H, P,
        zero_padding, _pn(xs, T and P), _stream(stream)))


def moe_permute_fp8(x, ld_x, slot_pos, sorted_ids, num_tokens_post_padded, T, k, H, P, zero_padding, q, s,
                    stream=None):
    return _check("moe_permute_fp8", load().moe_permute_fp8(
        _pn(x, T), ld_x, _pn(slot_pos, T), _pn(sorted_ids, T and P), _p(num_tokens_post_padded), T, k, H, P,
        zero_padding, _pn(q, T and P), _pn(s, T and P), _stream(stream)))


def moe_permute_backward(row_type, dxs, slot_pos, T, k, H, P, dx, ld_dx, stream=None):
    return _check("moe_permute_backward", load().moe_permute_backward(
        row_type, _pn(dxs, T and P), _pn(slot_pos, T), T, k, H, P, _pn(dx, T), ld_dx, _stream(stream)))


def moe_unpermute(row_type, ys, slot_pos, topk_weights, T, k, H, P, out, ld_out, stream=None):
    return _check("moe_unpermute", load().moe_unpermute(
        row_type, _pn(ys, T and P), _pn(slot_pos, T), _p(topk_weights), T, k, H, P, _pn(out, T), ld_out,
        _stream(stream)))


def moe_unpermute_backward(row_type, dout, ld_dout, ys, slot_pos, topk_weights, sorted_ids, num_tokens_post_padded,
                           T, k, H, P, zero_padding, dys, dweights, stream=None):
    return _check("moe_unpermute_backward", load().moe_unpermute_backward(
        row_type, _pn(dout, T), ld_dout, _pn(ys, T and P), _pn(slot_pos, T), _p(topk_weights),
        _pn(sorted_ids, T and P), _p(num_tokens_post_padded), T, k, H, P, zero_padding, _pn(dys, T and P),
        _pn(dweights, T), _stream(stream)))


def moe_gemm_fp8_block(A, a_scale, a_scale_by_block, B, b_scale, M, N, K, E, block_m, sorted_expert_ids,
                       num_tokens_post_padded, out_type, D, ld_d, ws, ws_bytes, stream=None):
    return _check("moe_gemm_fp8_block", load().moe_gemm_fp8_block(
        _pn(A, M), _pn(a_scale, M), a_scale_by_block, _p(B), _p(b_scale), M, N, K, E, block_m,
        _pn(sorted_expert_ids, M), _p(num_tokens_post_padded), out_type, _pn(D, M), ld_d, _p(ws), ws_bytes,
        _stream(stream)))


def moe_wgrad_fp8_block(A, a_scale, B, b_scale, P, M, N, E, expert_counts, D, accumulate, ws, ws_bytes, stream=None):
    return _check("moe_wgrad_fp8_block", load().moe_wgrad_fp8_block(
        _pn(A, P, ws), _pn(a_scale, P, ws), _pn(B, P, ws), _pn(b_scale, P, ws), P, M, N, E, _p(expert_counts), _p(D),
        accumulate, _p(ws), ws_bytes, _stream(stream)))


def moe_quantize_fp8_act_t(X, ld_x, R, C, sorted_ids, S, k, num_rows, q, ld_q, s, stream=None):
    return _check("moe_quantize_fp8_act_t", load().moe_quantize_fp8_act_t(
        _pn(X, R), ld_x, R, C, _p(sorted_ids), S, k, _p(num_rows), _pn(q, R), ld_q, _pn(s, R), _stream(stream)))


def moe_block_norm(row_type, h, residual, gate, gate_kind, w_post, w_pre, T, H, scale, weight_offset, eps, y, z,
                   rstd_h, rstd_y, stream=None):
    return _check("moe_block_norm", load().moe_block_norm(
        row_type, _pn(h, T), _pn(residual, T), _pn(gate, T), gate_kind, _p(w_post), _p(w_pre), T, H, scale,
        weight_offset, eps, _pn(y, T), _pn(z, T), _p(rstd_h), _p(rstd_y), _stream(stream)))


def moe_block_norm_workspace_size(T, H) -> int:
    return load().moe_block_norm_workspace_size(T, H)


def moe_block_norm_backward(row_type, h, residual, gate, gate_kind, w_post, w_pre, rstd_h, rstd_y, dy, dz, T, H, scale,
                            weight_offset, d_residual, dh, dgate, dw_post, dw_pre, ws, ws_bytes, stream=None):
    gates = H if gate_kind == MOE_GATE_CHANNEL else T  # (without rows, a column's gate and its gradient are still used)
    return _check("moe_block_norm_backward", load().moe_block_norm_backward(
        row_type, _pn(h, T), _pn(residual, T), _pn(gate, gates), gate_kind, _p(w_post), _p(w_pre), _pn(rstd_h, T),
        _pn(rstd_y, T), _pn(dy, T), _pn(dz, T), T, H, scale, weight_offset, _pn(d_residual, T), _pn(dh, T),
        _pn(dgate, gates), _p(dw_post), _p(dw_pre), _p(ws), ws_bytes, _stream(stream)))


class MoETrain:
    """Owns the training workspace of one bf16 layer shape: forward(), then backward()."""

    def __init__(self, T, H, I, E, k, device="cuda", options=None):
        import torch
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.options = options
        self.ws_bytes = moe_train_workspace_size(T, H, I, E, k)
        if self.ws_bytes == 0:
            raise MoEError("moe_train_workspace_size", MOE_ERR_INVALID_ARG)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def forward(self, x, w, out, stream=None):
        moe_fused_forward_train(x, w["W_router"], w.get("bias"), w["W_gate_up"], w["W_down"], self.T, self.H, self.I,
                                self.E, self.k, out, self.ws, self.ws_bytes, self.options, stream)
        return out

    def backward(self, x, w, dout, stream=None):
        """Returns dict dx (bf16), dW_gate_up, dW_down, dW_router, dbias (fp32)."""
        import torch
        dev = x.device
        g = {"dx": torch.empty(self.T, self.H, dtype=torch.bfloat16, device=dev),
             "dW_gate_up": torch.empty(self.E, 2 * self.I, self.H, dtype=torch.float32, device=dev),
             "dW_down": torch.empty(self.E, self.H, self.I, dtype=torch.float32, device=dev),
             "dW_router": torch.empty(self.E, self.H, dtype=torch.float32, device=dev),
             "dbias": torch.empty(self.E, dtype=torch.float32, device=dev)}
        moe_fused_backward(x, w["W_router"], w.get("bias"), w["W_gate_up"], w["W_down"], dout, self.T, self.H, self.I,
                           self.E, self.k, g["dx"], g["dW_gate_up"], g["dW_down"], g["dW_router"], g["dbias"], self.ws,
                           self.ws_bytes, self.options, stream)
        return g

    def status(self, stream=None) -> int:
        return moe_workspace_status(self.ws, stream)


# ------------------------------------------------------------- conveniences

_row_types = {}  # of torch's types, filled at the first use


def _row_type(dtype):
    if not _row_types:
        import torch
        _row_types.update({torch.bfloat16: MOE_ROW_BF16, torch.float16: MOE_ROW_FP16, torch.float32: MOE_ROW_FP32})
    row_type = _row_types.get(dtype)
    if row_type is None:
        raise TypeError(f"rows are bf16, fp16 or fp32, not {dtype}")
    return row_type


def _expect(name, t, shape, *dtypes):
    """t (None passes) is contiguous, of that shape and of one of those types."""
    if t is None:
        return
    if t.shape != shape or not t.is_contiguous():  # (a torch.Size is a tuple)
        raise ValueError(f"{name}: expected contiguous {tuple(shape)}, got {tuple(t.shape)} with strides {t.stride()}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")


def _on_gpu(owner, **tensors):
    """The tensors (None passes) are on the GPU of `owner`, a tensor of the object whose method is called: a
    kernel is given their addresses.  Checked last, right before a launch."""
    gpu = owner.get_device()  # (-1: not on a GPU)
    for t in tensors.values():
        if t is not None and t.get_device() != gpu:
            break
    else:
        if gpu >= 0:
            return
    for name, t in tensors.items():
        if t is not None and (gpu < 0 or t.get_device() != gpu):
            raise ValueError(f"{name} is on {t.device}, what belongs to the operator on {owner.device}: "
                             "both have to be on one GPU")


def _on(stream):
    """Context in which torch allocates and launches on `stream` (None: the current stream)."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _output(name, t, shape, dtype, device, stream):
    """t after its checks, or a new tensor that belongs to the stream that will write it."""
    if t is not None:
        _expect(name, t, shape, dtype)
        return t
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _codes():
    import torch
    return torch.uint8, torch.float8_e4m3fn


class TokenExchange:
    """Owns the maps of one routing shape (T tokens, k of E experts, blocks of block_m rows): sort(),
    then rows to the experts' order and back, with gradients.

    After sort(): sorted_ids, sorted_weights, expert_ids, num_tokens_post_padded, expert_counts, slot_pos
    and num_left_out (see moe_align_sort_drop in include/moe.h); P is the number of sorted rows to allocate.
    """

    def __init__(self, T, k, E, block_m=128, device="cuda"):
        import torch
        self.T, self.k, self.E, self.block_m = T, k, E, block_m
        self.P, nb = moe_align_sort_sizes(T, k, E, block_m)
        i32 = dict(dtype=torch.int32, device=device)
        self.sorted_ids, self.slot_pos = torch.empty(self.P, **i32), torch.empty(T * k, **i32)
        self.expert_ids, self.expert_counts = torch.empty(nb, **i32), torch.empty(E, **i32)
        self.num_tokens_post_padded, self.num_left_out = torch.empty(1, **i32), torch.empty(1, **i32)
        self.sorted_weights = torch.empty(self.P, dtype=torch.float32, device=device)
        self.ws_bytes = moe_align_sort_workspace_size(T, k, E)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.weights = None

    def sort(self, topk_ids, topk_weights, stream=None):
        """topk_ids int32 [T][k] (outside [0, E): the slot is left out, and counted in num_left_out),
        topk_weights fp32 [T][k]: kept, for unpermute and its gradient."""
        import torch
        _expect("topk_ids", topk_ids, (self.T, self.k), torch.int32)
        _expect("topk_weights", topk_weights, (self.T, self.k), torch.float32)
        _on_gpu(self.slot_pos, topk_ids=topk_ids, topk_weights=topk_weights)
        moe_align_sort_drop(topk_ids, topk_weights, self.T, self.k, self.E, self.block_m, self.sorted_ids,
                            self.sorted_weights, self.expert_ids, self.num_tokens_post_padded, self.expert_counts,
                            self.slot_pos, self.num_left_out, self.ws, self.ws_bytes, stream)
        self.weights = topk_weights

    def check_sorted(self):
        """Raises before the first sort(): the maps are unwritten memory until then."""
        if self.weights is None:
            raise ValueError("the exchange has no routing yet: sort() comes first")

    def segment_counts(self, stream=None):
        """Rows of each expert's segment, for moe_wgrad_fp8_block, which starts an expert after ceil(count / 128)
        blocks of 128 of each one before it: with larger sort blocks a segment's padding may hold whole blocks of
        128 (zero codes, which add nothing), so the counts are rounded up to the sort's blocks."""
        if self.block_m <= 128:
            return self.expert_counts
        with _on(stream):
            return (self.expert_counts + (self.block_m - 1)) // self.block_m * self.block_m

    def _rows(self, x):
        shape = x.shape
        if len(shape) != 2 or shape[0] != self.T or (shape[1] > 1 and x.stride(1) != 1):
            raise ValueError(f"expected {self.T} rows with contiguous elements, got {tuple(shape)}")
        # (a single row's stride means nothing to torch, which may give any)
        return shape[1], shape[1] if self.T == 1 else x.stride(0)

    def _token_rows(self, name, t, H, dtype, device, stream):
        """Token rows to write [T][H]: t (rows may be strided) after its checks, or new."""
        t = _output(name, None, (self.T, H), dtype, device, stream) if t is None else t
        h, ld = self._rows(t)
        if h != H or t.dtype != dtype:
            raise ValueError(f"{name}: expected {dtype} rows of {H}, got {t.dtype} rows of {h}")
        return t, ld

    def _sorted(self, ys):
        shape = ys.shape
        if len(shape) != 2 or shape[0] != self.P or not ys.is_contiguous():
            raise ValueError(f"expected {self.P} contiguous sorted rows, got {tuple(shape)}")
        return shape[1]

    def permute(self, x, xs=None, zero_padding=True, stream=None):
        """x [T][H] -> sorted rows [P][H]."""
        H, ld = self._rows(x)
        xs = _output("xs", xs, (self.P, H), x.dtype, x.device, stream)
        row_type = _row_type(x.dtype)
        _on_gpu(self.slot_pos, x=x, xs=xs)
        self.check_sorted()
        moe_permute(row_type, x, ld, self.slot_pos, self.sorted_ids, self.num_tokens_post_padded, self.T,
                    self.k, H, self.P, int(zero_padding), xs, stream)
        return xs

    def permute_fp8(self, x, q=None, s=None, zero_padding=True, stream=None):
        """x [T][H] bf16 -> e4m3 codes [P][H] (uint8) and scales by block [H/128][P]."""
        import torch
        H, ld = self._rows(x)
        if x.dtype != torch.bfloat16:
            raise TypeError("permute_fp8 takes bf16 rows")
        if q is not None:
            _expect("q", q, (self.P, H), *_codes())
        else:
            q = _output("q", None, (self.P, H), torch.uint8, x.device, stream)
        s = _output("s", s, (H // 128, self.P), torch.float32, x.device, stream)
        _on_gpu(self.slot_pos, x=x, q=q, s=s)
        self.check_sorted()
        moe_permute_fp8(x, ld, self.slot_pos, self.sorted_ids, self.num_tokens_post_padded, self.T, self.k, H, self.P,
                        int(zero_padding), q, s, stream)
        return q, s

    def unpermute(self, ys, out=None, weights=True, stream=None):
        """Sorted rows [P][H] -> [T][H], each token's rows summed with its top-k weights (or 1)."""
        H = self._sorted(ys)
        out, ld = self._token_rows("out", out, H, ys.dtype, ys.device, stream)
        row_type = _row_type(ys.dtype)
        _on_gpu(self.slot_pos, ys=ys, out=out)
        self.check_sorted()
        moe_unpermute(row_type, ys, self.slot_pos, self.weights if weights else None, self.T, self.k, H,
                      self.P, out, ld, stream)
        return out

    def unpermute_backward(self, dout, ys, zero_padding=True, stream=None):
        """Gradients of unpermute: (dys [P][H], dweights [T][k] fp32)."""
        import torch
        H, ld = self._rows(dout)
        _expect("ys", ys, (self.P, H), dout.dtype)
        dys = _output("dys", None, (self.P, H), ys.dtype, ys.device, stream)
        dw = _output("dweights", None, (self.T, self.k), torch.float32, ys.device, stream)
        row_type = _row_type(ys.dtype)
        _on_gpu(self.slot_pos, dout=dout, ys=ys)
        self.check_sorted()
        moe_unpermute_backward(row_type, dout, ld, ys, self.slot_pos, self.weights, self.sorted_ids,
                               self.num_tokens_post_padded, self.T, self.k, H, self.P, int(zero_padding), dys, dw,
                               stream)
        return dys, dw

    def permute_backward(self, dxs, dx=None, stream=None):
        """Gradient of permute: sorted rows [P][H] -> [T][H]."""
        H = self._sorted(dxs)
        dx, ld = self._token_rows("dx", dx, H, dxs.dtype, dxs.device, stream)
        row_type = _row_type(dxs.dtype)
        _on_gpu(self.slot_pos, dxs=dxs, dx=dx)
        self.check_sorted()
        moe_permute_backward(row_type, dxs, self.slot_pos, self.T, self.k, H, self.P, dx, ld, stream)
        return dx


class FusedMoE:
    """Owns the workspace for one layer shape and calls moe_fused_forward.

    weights: dict with W_router, bias (or None), W_gate_up, W_down (CUDA
    tensors); for FP8 also w1_scale, w2_scale and e4m3 (uint8) weight stacks.
    """

    def __init__(self, dtype, T, H, I, E, k, block_m=0, split_k=0, device="cuda", host_staging=False, options=None):
        import torch
        self.dtype, self.T, self.H, self.I, self.E, self.k = dtype, T, H, I, E, k
        self.options = options  # None (library defaults) or an Options
        self.block_m, self.split_k = block_m, split_k
        self.plan = moe_plan(dtype, T, H, I, E, k, block_m, split_k)
        self.ws_bytes = moe_fused_workspace_size(dtype, T, H, I, E, k, block_m, split_k)
        if self.ws_bytes == 0:
            raise MoEError("moe_fused_workspace_size", MOE_ERR_INVALID_ARG)
        extra = moe_host_staging_bytes(T, H) if host_staging else 0
        self.ws = torch.empty(self.ws_bytes + extra, dtype=torch.uint8, device=device)
        self.layout = moe_workspace_layout(dtype, T, H, I, E, k, block_m, split_k)

    def __call__(self, x, w, out, stream=None, options=None):
        """One forward; `options` (an Options) overrides the layer's own for this call."""
        opts = options if options is not None else self.options
        if opts is None:
            moe_fused_forward(self.dtype, x, w["W_router"], w.get("bias"), w["W_gate_up"], w.get("w1_scale"),
                              w["W_down"], w.get("w2_scale"), self.T, self.H, self.I, self.E, self.k, self.block_m,
                              self.split_k, out, self.ws, self.ws_bytes, stream)
        else:
            moe_fused_forward_ex(self.dtype, x, w["W_router"], w.get("bias"), w["W_gate_up"], w.get("w1_scale"),
                                 w["W_down"], w.get("w2_scale"), self.T, self.H, self.I, self.E, self.k, self.block_m,
                                 self.split_k, out, self.ws, self.ws_bytes, opts, stream)
        return out

    def capture(self, x, w, out, options=None):
        """A CUDA graph of one forward on these buffers (x, the weights, out and the workspace stay
        bound to it): graph.replay() reruns the whole layer, every kernel of the call, with one
        launch from the host -- for shapes where the host's per-call work would outlast the GPU's.
        The library allocates nothing and never synchronises, so a call is capturable as it is."""
        import torch
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self(x, w, out, options=options)  # outside the capture: the per-device launch limits are read here
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            self(x, w, out, options=options)
        return graph

    def forward_host(self, x_host, w, out_host, stream=None):
        moe_fused_forward_host(self.dtype, x_host, w["W_router"], w.get("bias"), w["W_gate_up"], w.get("w1_scale"),
                               w["W_down"], w.get("w2_scale"), self.T, self.H, self.I, self.E, self.k,
                               self.block_m, self.split_k, out_host, self.ws, self.ws.numel(), stream)
        return out_host

    def view(self, name, dtype, shape):
        """A tensor view of one intermediate buffer of the workspace (after a call)."""
        import torch
        off = getattr(self.layout, name)
        if off < 0:
            return None
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty(0, dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)

    def status(self, stream=None) -> int:
        return moe_workspace_status(self.ws, stream)


class FP8Weights:
    """Block-quantised weights of one product, [E][N][K] (E = 1: a dense layer): the e4m3 codes and the
    128 x 128 scales, and with `training` the transposed ones that the input gradient multiplies by.

    N and K are multiples of 128 (moe_quantize_fp8_weights).  Owns the products' workspace.  The constructor
    and update() write on `stream` as the products read on theirs: calls on different streams are the
    caller's to order."""

    def __init__(self, W, training=False, stream=None):
        import torch
        if W.dtype != torch.bfloat16 or W.dim() != 3 or not W.is_contiguous():
            raise ValueError("expected contiguous bf16 weights [E][N][K]")
        _on_gpu(W, W=W)
        E, N, K = self.E, self.N, self.K = W.shape
        self.training = training
        dev = W.device
        with _on(stream):
            self.ws = torch.zeros(MOE_GEMM_BLOCK_WS_BYTES, dtype=torch.uint8, device=dev)
            self.q = torch.empty(E, N, K, dtype=torch.uint8, device=dev)
            self.s = torch.empty(E, N // 128, K // 128, dtype=torch.float32, device=dev)
            if training:
                self.qt = torch.empty(E, K, N, dtype=torch.uint8, device=dev)
                self.st = torch.empty(E, K // 128, N // 128, dtype=torch.float32, device=dev)
        self.update(W, stream)

    def update(self, W, stream=None):
        """Quantise the weights anew (after an optimiser step), in place: products enqueued before on the same
        stream still read the old ones."""
        import torch
        _expect("W", W, (self.E, self.N, self.K), torch.bfloat16)
        _on_gpu(self.ws, W=W)
        moe_quantize_fp8_weights(W, self.E * self.N, self.K, self.q, self.s, stream)
        if self.training:  # the same blocks, transposed: the same codes and scales
            with _on(stream):
                self.qt.copy_(self.q.transpose(1, 2))
                self.st.copy_(self.s.transpose(1, 2))

    def _check_exchange(self, exchange):
        if (exchange is None and self.E != 1) or (exchange is not None and exchange.E != self.E):
            raise ValueError(f"{self.E} experts take sorted rows and the exchange of {self.E} experts that sorted them")

    def _product(self, a, a_scale, by_block, q, s, N, K, exchange, out, out_dtype, stream):
        import torch
        shape = a.shape
        if len(shape) != 2 or shape[1] != K or not a.is_contiguous():
            raise ValueError(f"expected contiguous rows of {K} codes, got {tuple(shape)}")
        M = shape[0]
        self._check_exchange(exchange)
        if exchange is not None and M != exchange.P:
            raise ValueError(f"expected the exchange's {exchange.P} sorted rows, got {M}")
        _expect("codes", a, (M, K), *_codes())
        KB = -(-K // 128)
        _expect("scales", a_scale, (KB, M) if by_block else (M, KB), torch.float32)
        dtype = out_dtype or (torch.bfloat16 if out is None else out.dtype)
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"products are bf16 or fp32, not {dtype}")
        out = _output("out", out, (M, N), dtype, a.device, stream)
        _on_gpu(self.ws, codes=a, scales=a_scale, out=out,
                exchange=None if exchange is None else exchange.slot_pos)
        if exchange is not None:
            exchange.check_sorted()
        g = (0, None, None) if exchange is None else (exchange.block_m, exchange.expert_ids,
                                                      exchange.num_tokens_post_padded)
        moe_gemm_fp8_block(a, a_scale, int(by_block), q, s, M, N, K, self.E, *g, _row_type(out.dtype), out,
                           N, self.ws, self.ws.numel(), stream)
        return out

    def product(self, a, a_scale, by_block=False, exchange=None, out=None, out_dtype=None, stream=None):
        """rows [M][K] (codes, scales) times W^T -> [M][N]; with an exchange (several experts need one), each
        sorted row times its expert's."""
        return self._product(a, a_scale, by_block, self.q, self.s, self.N, self.K, exchange, out, out_dtype, stream)

    def input_gradient(self, d, d_scale, by_block=False, exchange=None, out=None, out_dtype=None, stream=None):
        """rows [M][N] of an output gradient times W -> [M][K]."""
        if not self.training:
            raise ValueError("the input gradient needs FP8Weights(..., training=True)")
        return self._product(d, d_scale, by_block, self.qt, self.st, self.K, self.N, exchange, out, out_dtype, stream)

    def weight_gradient(self, d, d_scale, x, x_scale, exchange=None, out=None, accumulate=False, stream=None):
        """(d [N][P], x [K][P], as moe_quantize_fp8_act_t gives them) -> fp32 [E][N][K]."""
        import torch
        self._check_exchange(exchange)
        if d.dim() != 2:
            raise ValueError(f"expected codes [N][P], got {tuple(d.shape)}")
        P = d.shape[1]
        # each expert's blocks of 128 rows are its own: the sort's blocks have to be whole numbers of them
        if exchange is not None and (exchange.block_m % 128 or P < exchange.P):
            raise ValueError("the exchange's blocks have to be multiples of 128 rows, and P no less than its rows")
        for name, t, sc, rows in (("d", d, d_scale, self.N), ("x", x, x_scale, self.K)):
            _expect(name, t, (rows, P), *_codes())
            _expect(name + "_scale", sc, (P // 128, rows), torch.float32)
        if accumulate and out is None:
            raise ValueError("accumulate needs the gradients to add to")
        out = _output("out", out, (self.E, self.N, self.K), torch.float32, d.device, stream)
        _on_gpu(self.ws, d=d, d_scale=d_scale, x=x, x_scale=x_scale, out=out,
                exchange=None if exchange is None else exchange.slot_pos)
        if exchange is not None:
            exchange.check_sorted()
        counts = None if exchange is None else exchange.segment_counts(stream)
        moe_wgrad_fp8_block(d, d_scale, x, x_scale, d.shape[1], self.N, self.K, self.E, counts, out, int(accumulate),
                            self.ws, self.ws.numel(), stream)
        return out

    def status(self, stream=None) -> int:
        return moe_workspace_status(self.ws, stream)


class BlockNorm:
    """The norms before and after one block, with its gate and residual scale, for rows of one shape:
    forward(), then backward() (see moe_block_norm in include/moe.h).  Owns the kept statistics and the
    backward's workspace."""

    def __init__(self, T, H, gate_kind=MOE_GATE_NONE, scale=1.0, weight_offset=0.0, eps=1e-6, device="cuda"):
        import torch
        self.T, self.H, self.gate_kind = T, H, gate_kind
        self.scale, self.weight_offset, self.eps = scale, weight_offset, eps
        self.rstd_h, self.rstd_y = (torch.empty(T, dtype=torch.float32, device=device) for _ in range(2))
        self.kept = False, False  # the norms (after, before) whose statistics the last forward() has left
        self.ws_bytes = moe_block_norm_workspace_size(T, H)
        if self.ws_bytes == 0:
            raise MoEError("moe_block_norm_workspace_size", MOE_ERR_INVALID_ARG)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def _check(self, h, w_post, w_pre, gate, **rows):
        shape, columns, dtype = (self.T, self.H), (self.H,), h.dtype
        _expect("h", h, shape, dtype)
        for name, t in rows.items():
            _expect(name, t, shape, dtype)
        _expect("w_post", w_post, columns, dtype)
        _expect("w_pre", w_pre, columns, dtype)
        if self.gate_kind != MOE_GATE_NONE:
            _expect("gate", gate, self._gate_shape(), dtype)

    def _gate_shape(self):
        kind = self.gate_kind
        if kind == MOE_GATE_CHANNEL:
            return self.H,
        return None if kind == MOE_GATE_NONE else (self.T,) if kind == MOE_GATE_TOKEN else (self.T, self.H)

    def forward(self, h, residual, w_post=None, w_pre=None, gate=None, y=None, z=None, stream=None):
        """Returns (y, z): the residual stream after the block and the next block's input (None without w_pre)."""
        self._check(h, w_post, w_pre, gate, residual=residual)
        y = _output("y", y, h.shape, h.dtype, h.device, stream)
        if w_pre is not None:
            z = _output("z", z, h.shape, h.dtype, h.device, stream)
        row_type = _row_type(h.dtype)
        _on_gpu(self.ws, h=h, residual=residual, gate=gate, w_post=w_post, w_pre=w_pre, y=y, z=z)
        moe_block_norm(row_type, h, residual, gate, self.gate_kind, w_post, w_pre, self.T, self.H,
                       self.scale, self.weight_offset, self.eps, y, z, self.rstd_h, self.rstd_y, stream)
        self.kept = w_post is not None, w_pre is not None
        return y, z

    def backward(self, h, residual, dy, dz, w_post=None, w_pre=None, gate=None, stream=None):
        """Gradients of the last forward(), from its statistics: dict d_residual, dh, dgate, dw_post, dw_pre (None
        where there is no such input)."""
        import torch
        self._check(h, w_post, w_pre, gate, residual=residual, dy=dy, dz=dz)
        f32, shape = torch.float32, self._gate_shape()
        new = lambda name, shape, dtype: _output(name, None, shape, dtype, h.device, stream)  # noqa: E731
        g = {"d_residual": new("d_residual", h.shape, h.dtype), "dh": new("dh", h.shape, h.dtype),
             "dgate": None if shape is None else new("dgate", shape,
                                                     h.dtype if self.gate_kind == MOE_GATE_FULL else f32),
             "dw_post": None if w_post is None else new("dw_post", (self.H,), f32),
             "dw_pre": None if w_pre is None else new("dw_pre", (self.H,), f32)}
        row_type = _row_type(h.dtype)
        _on_gpu(self.ws, h=h, residual=residual, dy=dy, dz=dz, w_post=w_post, w_pre=w_pre, gate=gate)
        for name, w, kept in (("w_post", w_post, self.kept[0]), ("w_pre", w_pre, self.kept[1])):
            if w is not None and not kept:
                raise ValueError(f"{name}: no forward() with this norm has left its statistics")
        moe_block_norm_backward(row_type, h, residual, gate, self.gate_kind, w_post, w_pre, self.rstd_h,
                                self.rstd_y, dy, dz, self.T, self.H, self.scale, self.weight_offset, g["d_residual"],
                                g["dh"], g["dgate"], g["dw_post"], g["dw_pre"], self.ws, self.ws_bytes, stream)
        return g
