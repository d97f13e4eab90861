"""ctypes binding of libmoe.so (include/moe.h), same names as the C ABI.

Argument marshalling only: torch tensors are passed as device pointers, the
stream is torch's current stream, and tensor sizes are checked against the
shape before the call (the C side cannot see sizes). Every step runs in the
HIP library; if it is not built this module raises at import of the library.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK, MOE_E_INVALID, MOE_E_UNSUPPORTED, MOE_E_WORKSPACE, MOE_E_HIP = range(5)
MOE_F32, MOE_BF16, MOE_F8E4M3, MOE_F8E4M3_POW2, MOE_F4E2M1, MOE_BF16_TILED = 0, 1, 2, 3, 4, 5
MOE_ROWS_DIRECT, MOE_ROWS_GATHER, MOE_ROWS_SEGMENT = 0, 1, 2

MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED = 0, 1
MOE_ROPE_PLAIN, MOE_ROPE_LINEAR, MOE_ROPE_BASE, MOE_ROPE_PARTS = 0, 1, 2, 3

_STATUS = {1: "MOE_E_INVALID", 2: "MOE_E_UNSUPPORTED", 3: "MOE_E_WORKSPACE", 4: "MOE_E_HIP"}


class MoEError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class moe_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "n_routed", "n_groups", "topk_groups", "group_topn", "topk", "n_shared", "inter",
                 "batch_invariant")]

    @classmethod
    def of(cls, cfg) -> "moe_shape":
        return cls(cfg.T, cfg.d, cfg.n_routed, cfg.n_groups, cfg.topk_groups, cfg.group_topn, cfg.topk,
                   cfg.n_shared, cfg.inter, int(getattr(cfg, "batch_invariant", 0)))


class moe_heads(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("in_t", ctypes.c_int64), ("in_h", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_t", ctypes.c_int64), ("out_h", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class moe_rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("n_positions", ctypes.c_int32),
                ("table", ctypes.c_void_p)]


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()
_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_S = ctypes.POINTER(moe_shape)
_H, _R, _C, _D = (ctypes.POINTER(moe_heads), ctypes.POINTER(moe_rope), ctypes.POINTER(moe_kv_cache),
                  ctypes.c_double)

_SIGS = {
    "moe_route": [_S, _I, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_permute": [_S, _I, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P, ctypes.c_size_t, _P],
    "moe_permute_noalloc": [_S, _I, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P],
    "moe_permute_noalloc_max_scratch": [],
    "moe_grouped_ffn": [_S, _I, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P, ctypes.c_size_t, _P],
    "moe_ffn_gate_up": [_S, _I, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_ffn_down": [_S, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _P, ctypes.c_size_t, _P],
    "moe_combine": [_S, _I, _P, _P, _P, _P, _P, _P, _P],
    "moe_balance_stats": [_S, _P, _P, _I, ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_bias_update": [_S, _P, ctypes.c_float, _P, _P],
    "moe_quantize_weights": [_I, _I, _I, _I, _P, _P, _P, _P],
    "moe_quantize_weights_mxfp4": [_I, _I, _I, _I, _P, _P, _P, _P],
    "moe_tile_weights_bf16": [_I, _I, _I, _I, _P, _P, _P],
    "moe_ffn_gate_up_cache": [_S, _I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_combine_backward": [_S, _I, _P, _P, _P, _P, _I, _P, _P, _P],
    "moe_route_backward": [_S, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_transpose_weights_bf16": [_I, _I, _I, _P, _P, _P],
    "moe_ffn_backward_workspace_bytes": [_S, _I],
    "moe_ffn_backward": [_S, _I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_input_grad": [_S, _P, _P, _P, _P, _P, _P],
    "moe_transpose_bf16": [_I, _I, _I, _P, _P, _P],
    "moe_ffn_gate_up_cache_fp8": [_S, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_ffn_backward_fp8_workspace_bytes": [_S, _I, _I],
    "moe_ffn_backward_fp8": [_S, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                             ctypes.c_size_t, _P],
    "moe_rope_table": [_I, _I, _D, _I, _D, _D, _D, _D, _D, _P, _P],
    "moe_rotary": [_R, _I, _I, _I, _H, _H, _P, _P],
    "moe_rotary_backward": [_R, _I, _I, _I, _H, _H, _P, _P],
    "moe_kv_append": [_C, _R, _I, _I, _H, _H, _H, _P, _P, _P],
    "moe_prefix_attention_workspace_bytes": [_C, _I, _I, _I, _I, _I],
    "moe_prefix_attention": [_C, _I, _I, _I, _H, ctypes.c_float, _P, _I, _P, _I, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_causal_attention": [_I, _I, _I, _I, _P, _H, _H, _H, ctypes.c_float, _P, _P],
    "moe_causal_attention_backward": [_I, _I, _I, _I, _P, _H, _H, _H, _H, _H, ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
    "moe_causal_attention_backward_workspace_bytes": [_I, _I, _I, _I],
    "moe_layer_norm": [_I, _L, _I, _P, _L, _P, _P, ctypes.c_float, _P, _L, _P, _P, _P],
    "moe_layer_norm_backward": [_I, _L, _I, _P, _L, _P, _L, _P, _P, _P, _P, _L, _P, _L, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_layer_norm_backward_workspace_bytes": [_L, _I],
    "moe_workspace_bytes": [_S, _I],
    "moe_last_error": [],
    "moe_version": [],
}


def lib() -> ctypes.CDLL:
    """Load libmoe.so (once). Raises if the library has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is not built; run `python -m mixture_experts_layer_gate_amd.build`")
            L = ctypes.CDLL(LIB_PATH)
            for name, args in _SIGS.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = ctypes.c_size_t if name.endswith(("_bytes", "_max_scratch")) else ctypes.c_int
            L.moe_workspace_bytes.restype = ctypes.c_size_t
            L.moe_last_error.restype = ctypes.c_char_p
            L.moe_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


# MOE_SYNC_DEBUG=1: wait for the device after every call, so an asynchronous kernel error surfaces at the
# call that caused it
_SYNC_DEBUG = os.environ.get("MOE_SYNC_DEBUG") == "1"


def _check(status: int):
    if status != MOE_OK:
        raise MoEError(status, lib().moe_last_error().decode())
    if _SYNC_DEBUG:
        torch.cuda.synchronize()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object around it (3 us a call on the host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype in (torch.float8_e4m3fn, torch.uint8):
        return MOE_F8E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: Optional[torch.Tensor], numel: int, name: str):
    if t is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def moe_workspace_bytes(shape: moe_shape, gemm: int) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(shape), gemm))


def moe_route(shape: moe_shape, u, centroids, bias, topk_idx, topk_gate, expert_load, scores=None,
              workspace=None, stream=None):
    T, d, N, K = shape.T, shape.d, shape.n_routed, shape.topk
    _need(u, T * d, "u"); _need(centroids, N * d, "centroids"); _need(bias, N, "bias")
    _need(topk_idx, T * K, "topk_idx"); _need(topk_gate, T * K, "topk_gate"); _need(expert_load, N, "expert_load")
    _need(scores, T * N, "scores")
    _check(lib().moe_route(ctypes.byref(shape), _dt(u), _ptr(u), _ptr(centroids), _ptr(bias), _ptr(topk_idx),
                           _ptr(topk_gate), _ptr(expert_load), _ptr(scores), _ptr(workspace), _nbytes(workspace),
                           _stream(stream)))


def moe_permute(shape: moe_shape, topk_idx, u, expert_offsets, perm_token, row_of, a=None, a_dtype=None,
                a_scale=None, gather=1, workspace=None, stream=None):
    T, d, N, K = shape.T, shape.d, shape.n_routed, shape.topk
    _need(topk_idx, T * K, "topk_idx"); _need(expert_offsets, N + 1, "expert_offsets")
    _need(perm_token, T * K, "perm_token"); _need(row_of, T * K, "row_of")
    act = _dt(u) if u is not None else MOE_BF16
    if a is not None:
        rows = T * K if gather else T
        _need(u, T * d, "u"); _need(a, rows * d, "a")
        if a_dtype is None:
            a_dtype = _dt(a)
        if a_dtype in (MOE_F8E4M3, MOE_F8E4M3_POW2):
            _need(a_scale, rows * (d // 128), "a_scale")
    _check(lib().moe_permute(ctypes.byref(shape), act, _ptr(topk_idx), _ptr(u), _ptr(expert_offsets),
                             _ptr(perm_token), _ptr(row_of), _ptr(a), a_dtype if a_dtype is not None else act,
                             _ptr(a_scale), int(gather), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def moe_permute_noalloc(shape: moe_shape, topk_idx, u, expert_offsets, perm_token, row_of, a=None, a_dtype=None,
                        a_scale=None, gather=1, stream=None):
    """moe_permute on the library's static scratch: no workspace, nothing allocated."""
    T, d, N, K = shape.T, shape.d, shape.n_routed, shape.topk
    _need(topk_idx, T * K, "topk_idx"); _need(expert_offsets, N + 1, "expert_offsets")
    _need(perm_token, T * K, "perm_token"); _need(row_of, T * K, "row_of")
    act = _dt(u) if u is not None else MOE_BF16
    if a is not None:
        rows = T * K if gather else T
        _need(u, T * d, "u"); _need(a, rows * d, "a")
        if a_dtype is None:
            a_dtype = _dt(a)
        if a_dtype in (MOE_F8E4M3, MOE_F8E4M3_POW2):
            _need(a_scale, rows * (d // 128), "a_scale")
    _check(lib().moe_permute_noalloc(ctypes.byref(shape), act, _ptr(topk_idx), _ptr(u), _ptr(expert_offsets),
                                     _ptr(perm_token), _ptr(row_of), _ptr(a), a_dtype if a_dtype is not None else act,
                                     _ptr(a_scale), int(gather), _stream(stream)))


def _wscale_count(w: int, rows: int, cols: int) -> int:
    """Weight-scale entries of one [rows, cols] matrix: fp32 per 128x128 block, or E8M0 bytes per 1x32 (MXFP4,
    rows padded to whole 256-row tiles)."""
    return mx_rows(rows) * cols // 32 if w == MOE_F4E2M1 else (rows // 128) * (cols // 128)


def mx_rows(rows: int) -> int:
    """Rows of a matrix in the tiled E4M3 / MXFP4 weight layouts: whole 256-row tiles."""
    return -(-rows // 256) * 256


def moe_grouped_ffn(shape: moe_shape, w: int, n_experts: int, n_rows: int, expert_offsets, mode: int, row_src,
                    a, a_scale, a_rows: int, w_gate_up, w_gu_scale, w_down, w_d_scale, y, workspace=None,
                    stream=None):
    d, I = shape.d, shape.inter
    wdiv = 2 if w == MOE_F4E2M1 else 1            # MXFP4: two codes per byte
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(a, a_rows * d, "a")
    _need(w_gate_up, n_experts * 2 * I * d // wdiv, "w_gate_up")
    _need(w_down, n_experts * (mx_rows(d) if w in (MOE_F8E4M3, MOE_F4E2M1, MOE_BF16_TILED) else d) * I // wdiv,
          "w_down")
    _need(y, n_rows * d, "y")
    if mode == MOE_ROWS_GATHER:
        _need(row_src, n_rows, "row_src")
    if w in (MOE_F8E4M3, MOE_F4E2M1):
        _need(a_scale, a_rows * (d // 128), "a_scale")
        _need(w_gu_scale, n_experts * _wscale_count(w, 2 * I, d), "w_gu_scale")
        _need(w_d_scale, n_experts * _wscale_count(w, d, I), "w_d_scale")
    _check(lib().moe_grouped_ffn(ctypes.byref(shape), w, n_experts, n_rows, _ptr(expert_offsets), mode,
                                 _ptr(row_src), _ptr(a), _ptr(a_scale), a_rows, _ptr(w_gate_up), _ptr(w_gu_scale),
                                 _ptr(w_down), _ptr(w_d_scale), _dt(y), _ptr(y), _ptr(workspace),
                                 _nbytes(workspace), _stream(stream)))


def moe_ffn_gate_up(shape: moe_shape, w: int, n_experts: int, n_rows: int, expert_offsets, mode: int, row_src,
                    a, a_scale, a_rows: int, w_gate_up, w_gu_scale, h, h_scale=None, workspace=None, stream=None):
    d, I = shape.d, shape.inter
    wdiv = 2 if w == MOE_F4E2M1 else 1
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(a, a_rows * d, "a")
    _need(w_gate_up, n_experts * 2 * I * d // wdiv, "w_gate_up"); _need(h, n_rows * I, "h")
    if mode == MOE_ROWS_GATHER:
        _need(row_src, n_rows, "row_src")
    if w in (MOE_F8E4M3, MOE_F4E2M1):
        _need(a_scale, a_rows * (d // 128), "a_scale")
        _need(w_gu_scale, n_experts * _wscale_count(w, 2 * I, d), "w_gu_scale")
        _need(h_scale, n_rows * (I // 128), "h_scale")
    _check(lib().moe_ffn_gate_up(ctypes.byref(shape), w, n_experts, n_rows, _ptr(expert_offsets), mode,
                                 _ptr(row_src), _ptr(a), _ptr(a_scale), a_rows, _ptr(w_gate_up), _ptr(w_gu_scale),
                                 _ptr(h), _ptr(h_scale), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def moe_ffn_down(shape: moe_shape, w: int, n_experts: int, n_rows: int, expert_offsets, h, h_scale, w_down,
                 w_d_scale, y, workspace=None, stream=None):
    d, I = shape.d, shape.inter
    wdiv = 2 if w == MOE_F4E2M1 else 1
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(h, n_rows * I, "h")
    _need(w_down, n_experts * (mx_rows(d) if w in (MOE_F8E4M3, MOE_F4E2M1, MOE_BF16_TILED) else d) * I // wdiv,
          "w_down")
    _need(y, n_rows * d, "y")
    if w in (MOE_F8E4M3, MOE_F4E2M1):
        _need(h_scale, n_rows * (I // 128), "h_scale")
        _need(w_d_scale, n_experts * _wscale_count(w, d, I), "w_d_scale")
    _check(lib().moe_ffn_down(ctypes.byref(shape), w, n_experts, n_rows, _ptr(expert_offsets), _ptr(h),
                              _ptr(h_scale), _ptr(w_down), _ptr(w_d_scale), _dt(y), _ptr(y), _ptr(workspace),
                              _nbytes(workspace), _stream(stream)))


def moe_balance_stats(shape: moe_shape, scores, topk_idx, seq_len: int, alpha: float, f, P, loss, workspace,
                      stream=None):
    T, N, K = shape.T, shape.n_routed, shape.topk
    n_seq = -(-T // seq_len)
    _need(scores, T * N, "scores"); _need(topk_idx, T * K, "topk_idx")
    _need(f, n_seq * N, "f"); _need(P, n_seq * N, "P"); _need(loss, n_seq, "loss")
    _check(lib().moe_balance_stats(ctypes.byref(shape), _ptr(scores), _ptr(topk_idx), seq_len, ctypes.c_float(alpha),
                                   _ptr(f), _ptr(P), _ptr(loss), _ptr(workspace), _nbytes(workspace),
                                   _stream(stream)))


def moe_combine(shape: moe_shape, u, y_routed, row_of, topk_gate, y_shared, out, stream=None):
    T, d, K, Ns = shape.T, shape.d, shape.topk, shape.n_shared
    _need(u, T * d, "u"); _need(y_routed, T * K * d, "y_routed"); _need(row_of, T * K, "row_of")
    _need(topk_gate, T * K, "topk_gate"); _need(out, T * d, "out")
    if Ns:
        _need(y_shared, Ns * T * d, "y_shared")
    _check(lib().moe_combine(ctypes.byref(shape), _dt(u), _ptr(u), _ptr(y_routed), _ptr(row_of), _ptr(topk_gate),
                             _ptr(y_shared), _ptr(out), _stream(stream)))


def moe_bias_update(shape: moe_shape, expert_load, gamma: float, bias, stream=None):
    _need(expert_load, shape.n_routed, "expert_load"); _need(bias, shape.n_routed, "bias")
    _check(lib().moe_bias_update(ctypes.byref(shape), _ptr(expert_load), float(gamma), _ptr(bias),
                                 _stream(stream)))


def moe_quantize_weights(w, codes, scale, gate_up: bool, stream=None):
    """w [n, rows, cols] bf16 -> E4M3 codes in the tiled layout (n * ceil(rows/256)*256 * cols bytes) and fp32
    block scales [n, rows/128, cols/128] (gate_up: rows = 2I, gate rows then up rows)."""
    n, rows, cols = w.shape
    _need(codes, n * mx_rows(rows) * cols, "codes"); _need(scale, n * (rows // 128) * (cols // 128), "scale")
    _check(lib().moe_quantize_weights(n, rows, cols, int(gate_up), _ptr(w), _ptr(codes), _ptr(scale),
                                      _stream(stream)))


def moe_quantize_weights_mxfp4(w, codes, scales, gate_up: bool, stream=None):
    """w [n, rows, cols] bf16 -> MXFP4 in the tiled layout: codes n * ceil(rows/256)*256 * cols/2 bytes, scales
    n * ceil(rows/256)*256 * cols/32 bytes (gate_up: rows = 2I, gate rows then up rows)."""
    n, rows, cols = w.shape
    _need(codes, n * mx_rows(rows) * cols // 2, "codes"); _need(scales, n * mx_rows(rows) * (cols // 32), "scales")
    _check(lib().moe_quantize_weights_mxfp4(n, rows, cols, int(gate_up), _ptr(w), _ptr(codes), _ptr(scales),
                                            _stream(stream)))


def moe_tile_weights_bf16(w, out, gate_up: bool, stream=None):
    """w [n, rows, cols] bf16 -> out: the tiled layout of MOE_BF16_TILED (n * ceil(rows/256)*256 * cols bf16)."""
    n, rows, cols = w.shape
    _need(out, n * mx_rows(rows) * cols, "out")
    _check(lib().moe_tile_weights_bf16(n, rows, cols, int(gate_up), _ptr(w), _ptr(out), _stream(stream)))


# ---------------------------------------------------------------- backward

def moe_ffn_gate_up_cache(shape: moe_shape, w: int, n_experts: int, n_rows: int, expert_offsets, mode: int, row_src,
                          a, a_rows: int, w_gate_up, h, gu_cache, workspace=None, stream=None):
    d, I = shape.d, shape.inter
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(a, a_rows * d, "a")
    _need(h, n_rows * I, "h"); _need(gu_cache, n_rows * 2 * I, "gu_cache")
    if mode == MOE_ROWS_GATHER:
        _need(row_src, n_rows, "row_src")
    _check(lib().moe_ffn_gate_up_cache(ctypes.byref(shape), w, n_experts, n_rows, _ptr(expert_offsets), mode,
                                       _ptr(row_src), _ptr(a), a_rows, _ptr(w_gate_up), _ptr(h), _ptr(gu_cache),
                                       _ptr(workspace), _nbytes(workspace), _stream(stream)))


def moe_combine_backward(shape: moe_shape, d_out, y_routed, row_of, topk_gate, dy, d_gate, stream=None):
    T, d, K = shape.T, shape.d, shape.topk
    _need(d_out, T * d, "d_out"); _need(y_routed, T * K * d, "y_routed"); _need(row_of, T * K, "row_of")
    _need(topk_gate, T * K, "topk_gate"); _need(dy, (T * K + shape.n_shared * T) * d, "dy")
    _need(d_gate, T * K, "d_gate")
    _check(lib().moe_combine_backward(ctypes.byref(shape), _dt(d_out), _ptr(d_out), _ptr(y_routed), _ptr(row_of),
                                      _ptr(topk_gate), _dt(dy), _ptr(dy), _ptr(d_gate), _stream(stream)))


def moe_route_backward(shape: moe_shape, u, centroids, scores, topk_idx, d_gate, expert_offsets, perm_token, row_of,
                       du_router, d_centroids, workspace, stream=None):
    T, d, N, K = shape.T, shape.d, shape.n_routed, shape.topk
    _need(u, T * d, "u"); _need(centroids, N * d, "centroids"); _need(scores, T * N, "scores")
    _need(du_router, T * d, "du_router"); _need(d_centroids, N * d, "d_centroids")
    _check(lib().moe_route_backward(ctypes.byref(shape), _dt(u), _ptr(u), _ptr(centroids), _ptr(scores),
                                    _ptr(topk_idx), _ptr(d_gate), _ptr(expert_offsets), _ptr(perm_token),
                                    _ptr(row_of), _ptr(du_router), _ptr(d_centroids), _ptr(workspace),
                                    _nbytes(workspace), _stream(stream)))


def moe_transpose_weights_bf16(w, out, stream=None):
    """w [n, rows, cols] bf16 -> out: W^T [n, cols, rows] in the tiled layout (n * ceil(cols/256)*256 * rows)."""
    n, rows, cols = w.shape
    _need(out, n * mx_rows(cols) * rows, "out")
    _check(lib().moe_transpose_weights_bf16(n, rows, cols, _ptr(w), _ptr(out), _stream(stream)))


def moe_ffn_backward_workspace_bytes(shape: moe_shape, n_rows: int) -> int:
    return int(lib().moe_ffn_backward_workspace_bytes(ctypes.byref(shape), n_rows))


def moe_ffn_backward(shape: moe_shape, n_experts: int, n_rows: int, expert_offsets, mode: int, row_src, a,
                     a_rows: int, gu_cache, w_gate_up_t, w_down_t, dy, da, dw_gate_up, dw_down, workspace,
                     stream=None):
    d, I = shape.d, shape.inter
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(a, a_rows * d, "a")
    _need(gu_cache, n_rows * 2 * I, "gu_cache"); _need(dy, n_rows * d, "dy"); _need(da, n_rows * d, "da")
    _need(w_gate_up_t, n_experts * mx_rows(d) * 2 * I, "w_gate_up_t")
    _need(w_down_t, n_experts * mx_rows(I) * d, "w_down_t")
    _need(dw_gate_up, n_experts * 2 * I * d, "dw_gate_up"); _need(dw_down, n_experts * d * I, "dw_down")
    if mode == MOE_ROWS_GATHER:
        _need(row_src, n_rows, "row_src")
    _check(lib().moe_ffn_backward(ctypes.byref(shape), MOE_BF16_TILED, n_experts, n_rows, _ptr(expert_offsets), mode,
                                  _ptr(row_src), _ptr(a), a_rows, _ptr(gu_cache), _ptr(w_gate_up_t), _ptr(w_down_t),
                                  _ptr(dy), _ptr(da), _ptr(dw_gate_up), _ptr(dw_down), _ptr(workspace),
                                  _nbytes(workspace), _stream(stream)))


def moe_input_grad(shape: moe_shape, d_out, du_router, da, row_of, du, stream=None):
    T, d = shape.T, shape.d
    _need(d_out, T * d, "d_out"); _need(du, T * d, "du")
    _need(da, (T * shape.topk + shape.n_shared * T) * d, "da")
    _check(lib().moe_input_grad(ctypes.byref(shape), _ptr(d_out), _ptr(du_router), _ptr(da), _ptr(row_of), _ptr(du),
                                _stream(stream)))


# ---------------------------------------------------------------- FP8 backward

def moe_transpose_bf16(w, out, stream=None):
    """w [n, rows, cols] bf16 -> out [n, cols, rows] (row-major)."""
    n, rows, cols = w.shape
    _need(out, n * rows * cols, "out")
    _check(lib().moe_transpose_bf16(n, rows, cols, _ptr(w), _ptr(out), _stream(stream)))


def moe_ffn_gate_up_cache_fp8(shape: moe_shape, n_experts: int, n_rows: int, expert_offsets, mode: int, row_src,
                              a_codes, a_scale, a_rows: int, w_gate_up, w_gu_scale, h_codes, h_scale, gu_codes,
                              gu_scale, workspace=None, stream=None):
    d, I = shape.d, shape.inter
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(a_codes, a_rows * d, "a_codes")
    _need(a_scale, a_rows * (d // 128), "a_scale"); _need(h_codes, n_rows * I, "h_codes")
    _need(h_scale, n_rows * (I // 128), "h_scale"); _need(gu_codes, n_rows * 2 * I, "gu_codes")
    _need(gu_scale, n_rows * (2 * I // 128), "gu_scale")
    _need(w_gate_up, n_experts * mx_rows(2 * I) * d, "w_gate_up")
    if mode == MOE_ROWS_GATHER:
        _need(row_src, n_rows, "row_src")
    _check(lib().moe_ffn_gate_up_cache_fp8(ctypes.byref(shape), n_experts, n_rows, _ptr(expert_offsets), mode,
                                           _ptr(row_src), _ptr(a_codes), _ptr(a_scale), a_rows, _ptr(w_gate_up),
                                           _ptr(w_gu_scale), _ptr(h_codes), _ptr(h_scale), _ptr(gu_codes),
                                           _ptr(gu_scale), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def moe_ffn_backward_fp8_workspace_bytes(shape: moe_shape, n_rows: int, n_experts: int) -> int:
    return int(lib().moe_ffn_backward_fp8_workspace_bytes(ctypes.byref(shape), n_rows, n_experts))


def moe_ffn_backward_fp8(shape: moe_shape, n_experts: int, n_rows: int, expert_offsets, mode: int, row_src, a_codes,
                         a_scale, a_rows: int, gu_codes, gu_scale, w_gate_up_t, w_gate_up_t_scale, w_down_t,
                         w_down_t_scale, dy, da, dw_gate_up, dw_down, workspace, stream=None):
    d, I = shape.d, shape.inter
    _need(expert_offsets, n_experts + 1, "expert_offsets"); _need(a_codes, a_rows * d, "a_codes")
    _need(a_scale, a_rows * (d // 128), "a_scale"); _need(gu_codes, n_rows * 2 * I, "gu_codes")
    _need(gu_scale, n_rows * (2 * I // 128), "gu_scale")
    _need(w_gate_up_t, n_experts * mx_rows(d) * 2 * I, "w_gate_up_t")
    _need(w_gate_up_t_scale, n_experts * (d // 128) * (2 * I // 128), "w_gate_up_t_scale")
    _need(w_down_t, n_experts * mx_rows(I) * d, "w_down_t")
    _need(w_down_t_scale, n_experts * (I // 128) * (d // 128), "w_down_t_scale")
    _need(dy, n_rows * d, "dy"); _need(da, n_rows * d, "da")
    _need(dw_gate_up, n_experts * 2 * I * d, "dw_gate_up"); _need(dw_down, n_experts * d * I, "dw_down")
    if mode == MOE_ROWS_GATHER:
        _need(row_src, n_rows, "row_src")
    _check(lib().moe_ffn_backward_fp8(ctypes.byref(shape), n_experts, n_rows, _ptr(expert_offsets), mode,
                                      _ptr(row_src), _ptr(a_codes), _ptr(a_scale), a_rows, _ptr(gu_codes),
                                      _ptr(gu_scale), _ptr(w_gate_up_t), _ptr(w_gate_up_t_scale), _ptr(w_down_t),
                                      _ptr(w_down_t_scale), _ptr(dy), _ptr(da), _ptr(dw_gate_up), _ptr(dw_down),
                                      _ptr(workspace), _nbytes(workspace), _stream(stream)))


# ---------------------------------------------------------------- rotary positions, paged cache, attention

# These calls run once per layer and token in a decode step, so their checks are kept to a few tensor attributes.

_INT32_END = 1 << 31      # ctypes cuts a larger size off to 32 bits without a word


def _head_rows(x, out, name):
    """moe_heads of x [T, heads, head_dim] -> out (None: x is only read): any strides, channels contiguous."""
    shape, st = x.shape, x.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] (got {tuple(shape)})")
    if max(shape) >= _INT32_END:
        raise ValueError(f"{name} has 2^31 tokens, heads or channels, or more (got {tuple(shape)})")
    if st[2] != 1 and shape[2] > 1 and x.numel():
        raise ValueError(f"the channels of {name} must be contiguous")
    if out is None:
        return moe_heads(x.data_ptr(), st[0], st[1], None, st[0], st[1], shape[1])
    so = out.stride()
    if out.shape != shape:
        raise ValueError(f"{name}_out must have the shape of {name} (got {tuple(out.shape)})")
    if out.dtype != x.dtype:
        raise TypeError(f"{name}_out is {out.dtype}, {name} {x.dtype}")
    if so[2] != 1 and shape[2] > 1 and x.numel():
        raise ValueError(f"the channels of {name}_out must be contiguous")
    return moe_heads(x.data_ptr(), st[0], st[1], out.data_ptr(), so[0], so[1], shape[1])


def _ints(t, n, name):
    """Address of int32 t with at least n entries."""
    if t is None:
        return None
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32 (got {t.dtype})")
    if t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, needs {n}")
    return _addr(t)


def _addr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


def _rope_of(table, layout):
    shape = table.shape
    if table.dtype != torch.float32 or len(shape) != 3 or shape[2] != 2:
        raise ValueError("table must be fp32 [n_positions, rot_dim / 2, 2]")
    return moe_rope(2 * shape[1], layout, shape[0], _addr(table))


def _same_device(x, *others):
    """Every tensor on x's GPU, the current one."""
    d = x.get_device()
    if d < 0 or d != torch.cuda.current_device():
        raise ValueError(f"libmoe takes tensors of the current GPU (got one on {x.device})")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors on {x.device} and {t.device}")


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream`, from that stream's own: what is freed early is not handed to another stream's work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _act(t) -> int:
    """MOE_F32 or MOE_BF16; anything else is refused by the library."""
    return MOE_BF16 if t.dtype == torch.bfloat16 else MOE_F32 if t.dtype == torch.float32 else _dt(t)


def moe_rope_table(rot_dim: int, n_positions: int, base: float = 10000.0, scaling: int = MOE_ROPE_PLAIN,
                   factor: float = 1.0, orig_len: float = 0.0, slow: float = 1.0, fast: float = 32.0,
                   amplitude: float = 1.0, out=None, device="cuda", stream=None):
    """(cos, sin) of every position and channel pair: fp32 [n_positions, rot_dim / 2, 2] (allocated unless out)."""
    if out is None:
        if rot_dim <= 0 or rot_dim % 2 or n_positions <= 0:
            raise ValueError(f"rot_dim ({rot_dim}) must be positive and even, n_positions ({n_positions}) positive")
        out = _empty((n_positions, rot_dim // 2, 2), torch.float32, device, stream)
    if out.dtype != torch.float32:
        raise TypeError(f"the rotary table is fp32 (got {out.dtype})")
    _need(out, n_positions * rot_dim, "out")
    _same_device(out)
    _check(lib().moe_rope_table(rot_dim, n_positions, base, scaling, factor, orig_len, slow, fast, amplitude,
                                _ptr(out), _stream(stream)))
    return out


def _rotary(call, q, k, positions, table, q_out, k_out, layout, stream):
    T, _, D = q.shape
    if q_out is None or (k is not None and k_out is None):
        raise ValueError("every input needs its output")
    hq, hk = _head_rows(q, q_out, "q"), None
    if k is not None:
        hk = _head_rows(k, k_out, "k")
        if k.shape[0] != T or k.shape[2] != D or k.dtype != q.dtype:
            raise ValueError("k must be [tokens, heads, head_dim] with q's tokens, head_dim and dtype")
    pos, rope = _ints(positions, T, "positions"), _rope_of(table, layout)
    _same_device(q, k, positions, table, q_out, k_out)
    _check(call(rope, _act(q), T, D, hq, hk, pos, _stream(stream)))


def moe_rotary(q, k, positions, table, q_out, k_out=None, layout: int = MOE_ROPE_HALF, stream=None):
    """q [T, hq, D] -> q_out and k [T, hk, D] (or None) -> k_out, the leading 2 * table.shape[1] channels of every head
    rotated by table[positions[t]]. Any token and head strides; out may be the input itself."""
    _rotary(lib().moe_rotary, q, k, positions, table, q_out, k_out, layout, stream)


def moe_rotary_backward(dq, dk, positions, table, dq_out, dk_out=None, layout: int = MOE_ROPE_HALF, stream=None):
    """The gradients of moe_rotary's inputs from those of its outputs."""
    _rotary(lib().moe_rotary_backward, dq, dk, positions, table, dq_out, dk_out, layout, stream)


def _cache_of(k_cache, v_cache, k_scale, v_scale):
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must both be [n_pages, kv_heads, page_size, head_dim] of one dtype")
    n, h, p, d = shape
    dt = _act(k_cache)
    ks = vs = None
    if dt == MOE_F8E4M3:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None or t.dtype != torch.float32:
                raise ValueError(f"an E4M3 cache needs {name} as fp32 [n_pages, kv_heads, page_size]")
            _need(t, n * h * p, name)
        ks, vs = _addr(k_scale), _addr(v_scale)
    return moe_kv_cache(n, p, h, d, dt, _addr(k_cache), _addr(v_cache), ks, vs)


def moe_kv_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, positions=None, table=None,
                  layout: int = MOE_ROPE_HALF, q=None, q_out=None, stream=None):
    """Rotate k [T, kv_heads, D] by table[positions] (table None: no rotation) and write it and v to the cache rows
    slots [T] (page * page_size + row; outside the cache: not stored). With q [T, hq, D], also q -> q_out rotated.
    The cache: [n_pages, kv_heads, page_size, D] of k's dtype, or E4M3 codes (uint8 / float8_e4m3fn) with scales."""
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale)
    hk, hv, hq, rope = _head_rows(k, None, "k"), _head_rows(v, None, "v"), None, None
    T, D = k.shape[0], cache.head_dim
    if k.shape[2] != D or v.shape[0] != T or v.shape[2] != D or v.dtype != k.dtype:
        raise ValueError(f"k and v must be [tokens, heads, {D}] of one dtype")
    if q is not None:
        if q_out is None or table is None:
            raise ValueError("q needs q_out and a rotary table")
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != D or q.dtype != k.dtype:
            raise ValueError(f"q must be [{T} tokens, heads, {D}] in k's dtype")
        hq = _head_rows(q, q_out, "q")
    if table is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        rope = _rope_of(table, layout)
    sl, pos = _ints(slots, T, "slots"), _ints(positions, T, "positions")
    _same_device(k, v, slots, k_cache, v_cache, k_scale, v_scale, positions, table, q, q_out)
    _check(lib().moe_kv_append(cache, rope, _act(k), T, hk, hv, hq, pos, sl, _stream(stream)))


def moe_prefix_attention_workspace_bytes(k_cache, batch: int, q_len: int, q_heads: int, prefix_len: int,
                                         table_pages: int) -> int:
    n, h, p, d = k_cache.shape
    c = moe_kv_cache(n, p, h, d, _dt(k_cache), None, None, None, None)
    return int(lib().moe_prefix_attention_workspace_bytes(c, batch, q_len, q_heads, prefix_len, table_pages))


def moe_prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len: int, page_table, lens, out, q_len: int = 1,
                         scale: Optional[float] = None, k_scale=None, v_scale=None, lse=None, workspace=None,
                         stream=None):
    """Attention of q [batch * q_len, hq, D] -> out over the shared prefix (prefix_len tokens on prefix_pages) and each
    sequence's own tokens (lens [batch] on page_table [batch, table_pages]); scale defaults to 1 / sqrt(D). The work is cut
    for lens that average half of the table's width: a much wider table costs time.
    workspace: uint8 scratch (allocated for the call's stream unless given)."""
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale)
    if out is None:
        raise ValueError("out is needed")
    heads = _head_rows(q, out, "q")
    n, hq, D = q.shape
    if D != cache.head_dim:
        raise ValueError("q must be [batch * q_len, heads, head_dim] with the cache's head_dim")
    if q_len < 1 or n % q_len:
        raise ValueError(f"q has {n} tokens, not a multiple of q_len = {q_len}")
    B, cols, tab, ln = n // q_len, 0, None, None
    if page_table is not None:
        if page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError(f"page_table must be [batch = {B}, pages] (got {tuple(page_table.shape)})")
        cols = page_table.shape[1]
        if cols and lens is None:
            raise ValueError("page_table needs lens")
        tab, ln = _ints(page_table, B * cols, "page_table"), _ints(lens, B, "lens")
    if prefix_len > 0 and prefix_pages is None:
        raise ValueError("prefix_len > 0 needs prefix_pages")
    pre = _ints(prefix_pages, -(-prefix_len // cache.page_size), "prefix_pages")
    if lse is not None:
        if lse.dtype != torch.float32:
            raise TypeError("lse must be fp32")
        _need(lse, n * hq, "lse")
    _same_device(q, k_cache, v_cache, prefix_pages, page_table, lens, out, k_scale, v_scale, lse, workspace)
    L = lib()
    if workspace is None:
        nb = L.moe_prefix_attention_workspace_bytes(cache, B, q_len, hq, prefix_len, cols)
        workspace = _empty(max(nb, 256), torch.uint8, q.device, stream)
    _check(L.moe_prefix_attention(cache, _act(q), B, q_len, heads, D ** -0.5 if scale is None else scale, pre, prefix_len,
                                  tab, cols, ln, _addr(lse), _addr(workspace), _nbytes(workspace), _stream(stream)))


# ---------------------------------------------------------------- causal attention of packed sequences, layer norm

def _packed_heads(q, k, v):
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [tokens, heads, head_dim], k and v [tokens, kv_heads, head_dim]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError(f"q is {q.dtype}, k {k.dtype}, v {v.dtype}")


def _sequences(seq_start):
    if seq_start.dim() != 1 or seq_start.numel() < 1:
        raise ValueError("seq_start must be [n_seqs + 1]")
    if seq_start.numel() > _INT32_END:
        raise ValueError(f"seq_start has 2^31 sequences or more (got {seq_start.numel() - 1})")
    return seq_start.numel() - 1, _ints(seq_start, 1, "seq_start")


def _floats(t, n, name):
    """Address of fp32 t with at least n entries."""
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be fp32 (got {t.dtype})")
    _need(t, n, name)
    return _addr(t)


def moe_causal_attention(q, k, v, seq_start, out, scale: Optional[float] = None, lse=None, stream=None):
    """Causal attention of q [T, hq, D] -> out over k, v [T, hk, D]: sequence s is rows seq_start[s] .. seq_start[s + 1] - 1
    (int32 [n_seqs + 1], on the GPU); rows outside all sequences are left alone. lse: [T, hq] fp32 (the backward needs it).
    scale defaults to 1 / sqrt(D). Any token and head strides."""
    _packed_heads(q, k, v)
    if out is None:
        raise ValueError("out is needed")
    T, hq, D = q.shape
    n, starts = _sequences(seq_start)
    heads = _head_rows(q, out, "q"), _head_rows(k, None, "k"), _head_rows(v, None, "v")
    at = _floats(lse, T * hq, "lse")
    _same_device(q, k, v, seq_start, out, lse)
    _check(lib().moe_causal_attention(_act(q), T, D, n, starts, *heads, D ** -0.5 if scale is None else scale, at,
                                      _stream(stream)))


def moe_causal_attention_backward_workspace_bytes(T: int, head_dim: int, q_heads: int, kv_heads: int) -> int:
    """Bytes of scratch, 0 for sizes that the call refuses."""
    if max(T, head_dim, q_heads, kv_heads) >= _INT32_END:
        return 0
    return int(lib().moe_causal_attention_backward_workspace_bytes(T, head_dim, q_heads, kv_heads))


def moe_causal_attention_backward(d_out, q, k, v, out, lse, seq_start, dq, dk, dv, scale: Optional[float] = None,
                                  workspace=None, stream=None):
    """The gradients dq, dk and dv of moe_causal_attention's inputs, from d_out, its inputs, its out and its lse.
    workspace: uint8 scratch (allocated for the call's stream unless given)."""
    _packed_heads(q, k, v)
    if any(t is None for t in (d_out, out, lse, dq, dk, dv)):
        raise ValueError("d_out, out, lse, dq, dk and dv are needed")
    for t, name in ((out, "out"), (d_out, "d_out")):
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must have the shape and dtype of q (got {tuple(t.shape)}, {t.dtype})")
    T, hq, D = q.shape
    n, starts = _sequences(seq_start)
    heads = (_head_rows(q, dq, "q"), _head_rows(k, dk, "k"), _head_rows(v, dv, "v"), _head_rows(out, None, "out"),
             _head_rows(d_out, None, "d_out"))
    at = _floats(lse, T * hq, "lse")
    _same_device(q, k, v, out, d_out, lse, seq_start, dq, dk, dv, workspace)
    L = lib()
    if workspace is None:
        nb = L.moe_causal_attention_backward_workspace_bytes(T, D, hq, k.shape[1])
        workspace = _empty(max(nb, 256), torch.uint8, q.device, stream)
    _check(L.moe_causal_attention_backward(_act(q), T, D, n, starts, *heads, D ** -0.5 if scale is None else scale, at,
                                           _addr(workspace), _nbytes(workspace), _stream(stream)))


def _norm_rows(t, x, name):
    """(address, row stride) of t [rows, d], like x."""
    if t.shape != x.shape or t.dim() != 2:
        raise ValueError(f"{name} must be [rows, d] as x is (got {tuple(t.shape)})")
    if t.shape[1] >= _INT32_END:
        raise ValueError(f"{name} has 2^31 channels or more (got {t.shape[1]})")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} is {t.dtype}, x {x.dtype}")
    st = t.stride()
    if st[1] != 1 and t.shape[1] > 1 and t.numel():
        raise ValueError(f"the channels of {name} must be contiguous")
    return t.data_ptr(), st[0]


def moe_layer_norm(x, weight, bias, y, eps: float = 1e-5, mean=None, rstd=None, stream=None):
    """Layer norm of the rows of x [rows, d] -> y (any row strides; y may be x); weight and bias [d] fp32 or None;
    mean and rstd [rows] fp32 are written if given (the backward needs them)."""
    if y is None:
        raise ValueError("y is needed")
    rows, d = x.shape
    xs, ys = _norm_rows(x, x, "x"), _norm_rows(y, x, "y")
    vec = [_floats(t, n, m) for t, n, m in ((weight, d, "weight"), (bias, d, "bias"), (mean, rows, "mean"), (rstd, rows, "rstd"))]
    _same_device(x, weight, bias, y, mean, rstd)
    _check(lib().moe_layer_norm(_act(x), rows, d, *xs, *vec[:2], eps, *ys, *vec[2:], _stream(stream)))


def moe_layer_norm_backward_workspace_bytes(rows: int, d: int) -> int:
    """Bytes of scratch, 0 for sizes that the call refuses."""
    if d >= _INT32_END:
        return 0
    return int(lib().moe_layer_norm_backward_workspace_bytes(rows, d))


def moe_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, d_residual=None, workspace=None,
                            stream=None):
    """dx (of x [rows, d]), dweight and dbias ([d] fp32 or None) of moe_layer_norm from dy; d_residual: a gradient of x from
    elsewhere, added to dx. workspace: uint8 scratch (allocated for the call's stream unless given)."""
    if any(t is None for t in (mean, rstd, dx)):
        raise ValueError("mean, rstd and dx are needed")
    rows, d = x.shape
    ds, xs, os = _norm_rows(dy, x, "dy"), _norm_rows(x, x, "x"), _norm_rows(dx, x, "dx")
    rs = (None, 0) if d_residual is None else _norm_rows(d_residual, x, "d_residual")
    vec = [_floats(t, n, m) for t, n, m in ((weight, d, "weight"), (mean, rows, "mean"), (rstd, rows, "rstd"),
                                             (dweight, d, "dweight"), (dbias, d, "dbias"))]
    _same_device(x, dy, weight, mean, rstd, dx, dweight, dbias, d_residual, workspace)
    L = lib()
    if workspace is None:
        workspace = _empty(max(L.moe_layer_norm_backward_workspace_bytes(rows, d), 256), torch.uint8, x.device, stream)
    _check(L.moe_layer_norm_backward(_act(x), rows, d, *ds, *xs, *vec[:3], *rs, *os, *vec[3:], _addr(workspace),
                                     _nbytes(workspace), _stream(stream)))
