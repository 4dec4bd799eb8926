"""Python binding of libfp4bsa.so, the block-scaled FP4 quantized linear for B200.

Every function below has the name of the C entry point it calls (include/fp4bsa.h)
and only marshals arguments: tensors become device pointers, the current torch CUDA
stream becomes the stream argument, and a non-OK status raises FP4Error.  All
arithmetic runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or the device is not sm_100, the calls raise.

The helpers at the end (pack_weight, calibrate_act_global, quantize_act, linear, w4a8_linear,
w4a4_linear, gelu_quantize_act, linear_gelu_quant, linear_host, and around the attention
rope_table, qk_norm_rope, qk_norm_rope_quantize_heads, dequantize_heads, linear_residual,
attn_ranges, attn_bf16) allocate outputs and workspaces with torch and call the same entry points.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

from ._build import LIB as _LIB_PATH
from ._build import build

MXFP4, NVFP4 = 0, 1
_FMT = {"mxfp4": MXFP4, "nvfp4": NVFP4, MXFP4: MXFP4, NVFP4: NVFP4}

NORM_NONE, NORM_HEAD, NORM_TOKEN = 0, 1, 2
_NORM = {None: NORM_NONE, "none": NORM_NONE, "head": NORM_HEAD, "token": NORM_TOKEN, NORM_NONE: NORM_NONE,
         NORM_HEAD: NORM_HEAD, NORM_TOKEN: NORM_TOKEN}
ACT_NONE, ACT_GELU_TANH, ACT_SILU = 0, 1, 2
_ACT = {None: ACT_NONE, "none": ACT_NONE, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU, ACT_NONE: ACT_NONE,
        ACT_GELU_TANH: ACT_GELU_TANH, ACT_SILU: ACT_SILU}
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
_ROPE = {"interleaved": ROPE_INTERLEAVED, "half": ROPE_HALF, ROPE_INTERLEAVED: ROPE_INTERLEAVED, ROPE_HALF: ROPE_HALF}

STATUS = ["FP4_OK", "FP4_ERR_INVALID_ARG", "FP4_ERR_UNSUPPORTED_SHAPE", "FP4_ERR_MISALIGNED",
          "FP4_ERR_WORKSPACE", "FP4_ERR_ARCH", "FP4_ERR_CUDA", "FP4_ERR_TIMEOUT"]

# every symbol include/fp4bsa.h declares
EXPORTS = [
    "fp4_codes_bytes", "fp4_sf_bytes", "fp4_linear_workspace_bytes", "w4a8_workspace_bytes",
    "fp4_tensor_amax", "fp4_pack_weight", "fp4_quantize_act", "fp4_gemm", "fp4_linear",
    "w4a8_quantize_act", "w4a8_gemm", "w4a8_svd_linear", "fp4_sync_status", "fp4_status_string",
    "fp4_set_wait_timeout_ns", "fp4_linear_noalloc",
    "w4a4_workspace_bytes", "w4a4_quantize_act", "w4a4_gemm", "w4a4_svd_linear",
    "fp4_gelu_quantize_act", "fp4_gemm_gelu_quant", "fp4_linear_gelu_quant", "fp4_calibrate_act_global",
    "fp4_heads_codes_bytes", "fp4_heads_sf_bytes", "fp4_quantize_heads", "fp4_attn_scores",
    "fp4_heads_vt_codes_bytes", "fp4_heads_vt_sf_bytes", "fp4_quantize_heads_vt", "fp4_attn_softmax_quant",
    "fp4_attn_pv",
    "fp4_attn_fused",
    "fp4_attn_fused_trace",
    "fp4_gemm_residual", "fp4_linear_residual",
    "fp4_rope_table", "fp4_qk_norm_rope", "fp4_qk_norm_rope_quantize_heads", "fp4_dequantize_heads",
    "fp4_attn_bf16_workspace_bytes", "fp4_attn_bf16", "fp4_attn_ranges",
]


class FP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = STATUS[status] if 0 <= status < len(STATUS) else f"status {status}"
        super().__init__(f"{where}: {name}")


_lib = None


def lib():
    """Load libfp4bsa.so (it must have been built; see build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: run fp4_block_scaled_act_b200.build() first")
        L = ctypes.CDLL(_LIB_PATH)
        P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        D, F = ctypes.c_double, ctypes.c_float
        sig = {
            "fp4_codes_bytes": (SZ, [I, I64, I64]),
            "fp4_sf_bytes": (SZ, [I, I64, I64]),
            "fp4_linear_workspace_bytes": (SZ, [I, I64, I64, I64]),
            "w4a8_workspace_bytes": (SZ, [I64, I64, I64, I]),
            "fp4_tensor_amax": (I, [P, I64, P, P]),
            "fp4_pack_weight": (I, [I, P, I64, I64, P, P, P, P]),
            "fp4_calibrate_act_global": (I, [P, I64, P, P, P]),
            "fp4_quantize_act": (I, [I, P, I64, I64, P, P, P, P]),
            "fp4_gemm": (I, [I, P, P, I64, I64, I64, P, P, P, P, P, P, P]),
            "fp4_linear": (I, [I, P, I64, I64, I64, P, P, P, P, P, P, P, SZ, P]),
            "fp4_linear_noalloc": (I, [I, P, I64, I64, I64, P, P, P, P, P, P, P]),
            "w4a8_quantize_act": (I, [P, I64, I64, P, I, P, P, P, P]),
            "w4a4_workspace_bytes": (SZ, [I64, I64, I64, I]),
            "fp4_gelu_quantize_act": (I, [I, P, I64, I64, P, P, P, P]),
            "fp4_gemm_gelu_quant": (I, [I, P, P, I64, I64, I64, P, P, P, P, P, P, P, P, P]),
            "fp4_linear_gelu_quant": (I, [I, P, I64, I64, I64, P, P, P, P, P, P, P, P, P, SZ, P]),
            "w4a4_quantize_act": (I, [P, I64, I64, P, I, P, P, P, P]),
            "w4a4_gemm": (I, [P, P, P, I64, I64, I64, P, P, P, I, P, P, P]),
            "w4a4_svd_linear": (I, [P, I64, I64, I64, P, P, P, P, I, P, P, P, SZ, P]),
            "w4a8_gemm": (I, [P, P, P, I64, I64, I64, P, P, P, I, P, P, P]),
            "w4a8_svd_linear": (I, [P, I64, I64, I64, P, P, P, P, I, P, P, P, SZ, P]),
            "fp4_heads_codes_bytes": (SZ, [I, I64, I64, I64]),
            "fp4_heads_sf_bytes": (SZ, [I, I64, I64, I64]),
            "fp4_quantize_heads": (I, [I, P, I64, I64, I64, P, P, P, P]),
            "fp4_attn_scores": (I, [I, P, P, I64, P, P, I64, I64, I64, I64, P, P, P, P]),
            "fp4_heads_vt_codes_bytes": (SZ, [I, I64, I64, I64]),
            "fp4_heads_vt_sf_bytes": (SZ, [I, I64, I64, I64]),
            "fp4_quantize_heads_vt": (I, [I, P, I64, I64, I64, P, P, P, P]),
            "fp4_attn_softmax_quant": (I, [I, P, I64, I64, ctypes.c_float, P, P, P, P, P]),
            "fp4_attn_pv": (I, [I, P, P, P, I64, I64, P, P, P, I64, I64, I64, P, P, P]),
            "fp4_attn_fused": (I, [I, P, P, I64, P, P, I64, P, P, I64, I64, I64, ctypes.c_float, P, P, P, P, P, P,
                                   P]),
            "fp4_attn_fused_trace": (I, [I, P, P, I64, P, P, I64, P, P, I64, I64, I64, ctypes.c_float, P, P, P, P, P,
                                         P, I64, P, P, P, P]),
            "fp4_gemm_residual": (I, [I, P, P, I64, I64, I64, P, P, P, P, P, I, P, I64, P, P, P]),
            "fp4_linear_residual": (I, [I, P, I64, I64, I64, P, P, P, P, P, I, P, I64, P, P, P, SZ, P]),
            "fp4_rope_table": (I, [P, I64, I, P, D, D, I64, F, P, P]),
            "fp4_qk_norm_rope": (I, [P, I64, I64, P, I64, I64, I64, I64, I, P, P, F, P, I64, I, P, I64, P, I64, P]),
            "fp4_qk_norm_rope_quantize_heads": (I, [I, P, I64, I64, P, I64, I64, I64, I64, I, P, P, F, P, I64, I, P, P,
                                                    P, P, P, P, P]),
            "fp4_dequantize_heads": (I, [I, P, P, I64, I64, I64, P, P, I64, P]),
            "fp4_attn_bf16_workspace_bytes": (SZ, [I64, I64, I64, I64, I64]),
            "fp4_attn_bf16": (I, [P, I64, I64, P, I64, P, I64, I64, I64, I64, I64, F, F, P, I64, P, P, P, I64, P, P, SZ,
                                  P]),
            "fp4_attn_ranges": (I, [P, P, I64, I64, I64, I, P, P, P, P]),
            "fp4_sync_status": (I, [P]),
            "fp4_status_string": (ctypes.c_char_p, [I]),
            "fp4_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
            "fp4bsa_test_skip_iteration": (None, [I]),
            "fp4bsa_set_gemm_ctas": (None, [I]),
            "fp4bsa_set_stream_k": (None, [I]),
            "fp4bsa_set_pdl": (None, [I]),
            "fp4bsa_test_gelu_f32": (I, [P, I64, P, P]),
            "fp4bsa_clock_probe": (I, [P, I, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# ----------------------------------------------------------------------------- marshalling
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _rows_ptr(t) -> Optional[int]:
    """Pointer of a [T, H, D] tensor whose rows may lie apart (the caller passes its row stride)."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream=None):
    import torch

    if stream is None:
        # (the current stream's handle without a Stream object around it: a few microseconds a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str):
    if status != 0:
        raise FP4Error(status, where)


def _fmt(fmt) -> int:
    return _FMT[fmt]


# ----------------------------------------------------------------------------- entry points
def fp4_codes_bytes(fmt, rows: int, K: int) -> int:
    return lib().fp4_codes_bytes(_fmt(fmt), rows, K)


def fp4_sf_bytes(fmt, rows: int, K: int) -> int:
    return lib().fp4_sf_bytes(_fmt(fmt), rows, K)


def fp4_linear_workspace_bytes(fmt, M: int, K: int, N: int) -> int:
    return lib().fp4_linear_workspace_bytes(_fmt(fmt), M, K, N)


def w4a8_workspace_bytes(M: int, K: int, N: int, rank: int = 32) -> int:
    return lib().w4a8_workspace_bytes(M, K, N, rank)


def fp4_tensor_amax(x, n: int, amax_out, stream=None):
    _check(lib().fp4_tensor_amax(_ptr(x), n, _ptr(amax_out), _stream(stream)), "fp4_tensor_amax")


def fp4_calibrate_act_global(x, n: int, amax_inout, g_out, stream=None):
    _check(lib().fp4_calibrate_act_global(_ptr(x), n, _ptr(amax_inout), _ptr(g_out), _stream(stream)),
           "fp4_calibrate_act_global")


def fp4_pack_weight(fmt, w, N: int, K: int, w_codes, w_sf, w_global=None, stream=None):
    _check(lib().fp4_pack_weight(_fmt(fmt), _ptr(w), N, K, _ptr(w_codes), _ptr(w_sf), _ptr(w_global),
                                 _stream(stream)), "fp4_pack_weight")


def fp4_quantize_act(fmt, x, M: int, K: int, a_global, x_codes, x_sf, stream=None):
    _check(lib().fp4_quantize_act(_fmt(fmt), _ptr(x), M, K, _ptr(a_global), _ptr(x_codes), _ptr(x_sf),
                                  _stream(stream)), "fp4_quantize_act")


def fp4_gemm(fmt, a_codes, a_sf, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias, y,
             stream=None):
    _check(lib().fp4_gemm(_fmt(fmt), _ptr(a_codes), _ptr(a_sf), M, K, N, _ptr(w_codes), _ptr(w_sf),
                          _ptr(w_global), _ptr(a_global), _ptr(bias), _ptr(y), _stream(stream)), "fp4_gemm")


def fp4_linear(fmt, x, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias, y, workspace,
               ws_bytes: int, stream=None):
    _check(lib().fp4_linear(_fmt(fmt), _ptr(x), M, K, N, _ptr(w_codes), _ptr(w_sf), _ptr(w_global),
                            _ptr(a_global), _ptr(bias), _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)),
           "fp4_linear")


def fp4_linear_noalloc(fmt, x, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias, y,
                       stream=None):
    """fp4_linear without a workspace argument, for callers that cannot allocate device
    memory: the quantized activations use the library's built-in 16 MiB device array."""
    _check(lib().fp4_linear_noalloc(_fmt(fmt), _ptr(x), M, K, N, _ptr(w_codes), _ptr(w_sf), _ptr(w_global),
                                    _ptr(a_global), _ptr(bias), _ptr(y), _stream(stream)), "fp4_linear_noalloc")


def fp4_gelu_quantize_act(fmt, z, M: int, K: int, a_global, x_codes, x_sf, stream=None):
    _check(lib().fp4_gelu_quantize_act(_fmt(fmt), _ptr(z), M, K, _ptr(a_global), _ptr(x_codes), _ptr(x_sf),
                                       _stream(stream)), "fp4_gelu_quantize_act")


def fp4_gemm_gelu_quant(fmt, a_codes, a_sf, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias,
                        h_global, h_codes, h_sf, stream=None):
    _check(lib().fp4_gemm_gelu_quant(_fmt(fmt), _ptr(a_codes), _ptr(a_sf), M, K, N, _ptr(w_codes), _ptr(w_sf),
                                     _ptr(w_global), _ptr(a_global), _ptr(bias), _ptr(h_global), _ptr(h_codes),
                                     _ptr(h_sf), _stream(stream)), "fp4_gemm_gelu_quant")


def fp4_linear_gelu_quant(fmt, x, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias, h_global,
                          h_codes, h_sf, workspace, ws_bytes: int, stream=None):
    _check(lib().fp4_linear_gelu_quant(_fmt(fmt), _ptr(x), M, K, N, _ptr(w_codes), _ptr(w_sf), _ptr(w_global),
                                       _ptr(a_global), _ptr(bias), _ptr(h_global), _ptr(h_codes), _ptr(h_sf),
                                       _ptr(workspace), ws_bytes, _stream(stream)), "fp4_linear_gelu_quant")


def w4a8_quantize_act(x, M: int, K: int, l1, rank: int, x_e4m3, x_sf, u_pair, stream=None):
    _check(lib().w4a8_quantize_act(_ptr(x), M, K, _ptr(l1), rank, _ptr(x_e4m3), _ptr(x_sf), _ptr(u_pair),
                                   _stream(stream)), "w4a8_quantize_act")


def w4a8_gemm(x_e4m3, x_sf, u_pair, M: int, K: int, N: int, r_codes, r_sf, l2, rank: int, bias, y,
              stream=None):
    _check(lib().w4a8_gemm(_ptr(x_e4m3), _ptr(x_sf), _ptr(u_pair), M, K, N, _ptr(r_codes), _ptr(r_sf),
                           _ptr(l2), rank, _ptr(bias), _ptr(y), _stream(stream)), "w4a8_gemm")


def w4a8_svd_linear(x, M: int, K: int, N: int, r_codes, r_sf, l1, l2, rank: int, bias, y, workspace,
                    ws_bytes: int, stream=None):
    _check(lib().w4a8_svd_linear(_ptr(x), M, K, N, _ptr(r_codes), _ptr(r_sf), _ptr(l1), _ptr(l2), rank,
                                 _ptr(bias), _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)),
           "w4a8_svd_linear")


def w4a4_workspace_bytes(M: int, K: int, N: int, rank: int = 32) -> int:
    return lib().w4a4_workspace_bytes(M, K, N, rank)


def w4a4_quantize_act(x, M: int, K: int, l1, rank: int, x_codes, x_sf, u_pair, stream=None):
    _check(lib().w4a4_quantize_act(_ptr(x), M, K, _ptr(l1), rank, _ptr(x_codes), _ptr(x_sf), _ptr(u_pair),
                                   _stream(stream)), "w4a4_quantize_act")


def w4a4_gemm(x_codes, x_sf, u_pair, M: int, K: int, N: int, r_codes, r_sf, l2, rank: int, bias, y,
              stream=None):
    _check(lib().w4a4_gemm(_ptr(x_codes), _ptr(x_sf), _ptr(u_pair), M, K, N, _ptr(r_codes), _ptr(r_sf),
                           _ptr(l2), rank, _ptr(bias), _ptr(y), _stream(stream)), "w4a4_gemm")


def w4a4_svd_linear(x, M: int, K: int, N: int, r_codes, r_sf, l1, l2, rank: int, bias, y, workspace,
                    ws_bytes: int, stream=None):
    _check(lib().w4a4_svd_linear(_ptr(x), M, K, N, _ptr(r_codes), _ptr(r_sf), _ptr(l1), _ptr(l2), rank,
                                 _ptr(bias), _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)),
           "w4a4_svd_linear")


def fp4_heads_codes_bytes(fmt, T: int, H: int, D: int = 128) -> int:
    return lib().fp4_heads_codes_bytes(_fmt(fmt), T, H, D)


def fp4_heads_sf_bytes(fmt, T: int, H: int, D: int = 128) -> int:
    return lib().fp4_heads_sf_bytes(_fmt(fmt), T, H, D)


def fp4_quantize_heads(fmt, x, T: int, H: int, D: int, g, codes, sf, stream=None):
    _check(lib().fp4_quantize_heads(_fmt(fmt), _ptr(x), T, H, D, _ptr(g), _ptr(codes), _ptr(sf), _stream(stream)),
           "fp4_quantize_heads")


def fp4_attn_scores(fmt, q_codes, q_sf, T_q: int, k_codes, k_sf, T_kv: int, H: int, D: int, head: int, g_q, g_k,
                    s, stream=None):
    _check(lib().fp4_attn_scores(_fmt(fmt), _ptr(q_codes), _ptr(q_sf), T_q, _ptr(k_codes), _ptr(k_sf), T_kv, H, D,
                                 head, _ptr(g_q), _ptr(g_k), _ptr(s), _stream(stream)), "fp4_attn_scores")


def fp4_heads_vt_codes_bytes(fmt, T: int, H: int, D: int = 128) -> int:
    return lib().fp4_heads_vt_codes_bytes(_fmt(fmt), T, H, D)


def fp4_heads_vt_sf_bytes(fmt, T: int, H: int, D: int = 128) -> int:
    return lib().fp4_heads_vt_sf_bytes(_fmt(fmt), T, H, D)


def fp4_quantize_heads_vt(fmt, v, T: int, H: int, D: int, g, codes, sf, stream=None):
    _check(lib().fp4_quantize_heads_vt(_fmt(fmt), _ptr(v), T, H, D, _ptr(g), _ptr(codes), _ptr(sf),
                                       _stream(stream)), "fp4_quantize_heads_vt")


def fp4_attn_softmax_quant(fmt, s, T_q: int, T_kv: int, scale: float, p_global, stats, p_codes, p_sf,
                           stream=None):
    _check(lib().fp4_attn_softmax_quant(_fmt(fmt), _ptr(s), T_q, T_kv, float(scale), _ptr(p_global), _ptr(stats),
                                        _ptr(p_codes), _ptr(p_sf), _stream(stream)), "fp4_attn_softmax_quant")


def fp4_attn_pv(fmt, p_codes, p_sf, p_global, T_q: int, T_kv: int, vt_codes, vt_sf, v_global, H: int, D: int,
                head: int, stats, o, stream=None):
    _check(lib().fp4_attn_pv(_fmt(fmt), _ptr(p_codes), _ptr(p_sf), _ptr(p_global), T_q, T_kv, _ptr(vt_codes),
                             _ptr(vt_sf), _ptr(v_global), H, D, head, _ptr(stats), _ptr(o), _stream(stream)),
           "fp4_attn_pv")


def fp4_attn_fused(fmt, q_codes, q_sf, T_q: int, k_codes, k_sf, T_kv: int, vt_codes, vt_sf, H: int, D: int,
                   head: int, scale: float, g_q, g_k, g_v, p_global, stats, o, stream=None):
    _check(lib().fp4_attn_fused(_fmt(fmt), _ptr(q_codes), _ptr(q_sf), T_q, _ptr(k_codes), _ptr(k_sf), T_kv,
                                _ptr(vt_codes), _ptr(vt_sf), H, D, head, scale, _ptr(g_q), _ptr(g_k), _ptr(g_v),
                                _ptr(p_global), _ptr(stats), _ptr(o), _stream(stream)), "fp4_attn_fused")


def fp4_attn_fused_trace(fmt, q_codes, q_sf, T_q: int, k_codes, k_sf, T_kv: int, vt_codes, vt_sf, H: int, D: int,
                         head: int, scale: float, g_q, g_k, g_v, p_global, stats, o, trace_tile: int, trace_m,
                         trace_codes, trace_sf, stream=None):
    _check(lib().fp4_attn_fused_trace(_fmt(fmt), _ptr(q_codes), _ptr(q_sf), T_q, _ptr(k_codes), _ptr(k_sf), T_kv,
                                      _ptr(vt_codes), _ptr(vt_sf), H, D, head, scale, _ptr(g_q), _ptr(g_k),
                                      _ptr(g_v), _ptr(p_global), _ptr(stats), _ptr(o), trace_tile, _ptr(trace_m),
                                      _ptr(trace_codes), _ptr(trace_sf), _stream(stream)), "fp4_attn_fused_trace")


def fp4_gemm_residual(fmt, a_codes, a_sf, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias, act, gate,
                      gate_rows: int, residual, y, stream=None):
    _check(lib().fp4_gemm_residual(_fmt(fmt), _ptr(a_codes), _ptr(a_sf), M, K, N, _ptr(w_codes), _ptr(w_sf),
                                   _ptr(w_global), _ptr(a_global), _ptr(bias), _ACT[act], _ptr(gate), gate_rows,
                                   _ptr(residual), _ptr(y), _stream(stream)), "fp4_gemm_residual")


def fp4_linear_residual(fmt, x, M: int, K: int, N: int, w_codes, w_sf, w_global, a_global, bias, act, gate,
                        gate_rows: int, residual, y, workspace, ws_bytes: int, stream=None):
    _check(lib().fp4_linear_residual(_fmt(fmt), _ptr(x), M, K, N, _ptr(w_codes), _ptr(w_sf), _ptr(w_global),
                                     _ptr(a_global), _ptr(bias), _ACT[act], _ptr(gate), gate_rows, _ptr(residual),
                                     _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)), "fp4_linear_residual")


def fp4_rope_table(positions, T: int, axes: int, axis_dims, theta: float, factor: float, window: int,
                   amplitude: float, table, stream=None):
    dims = (ctypes.c_int64 * len(axis_dims))(*axis_dims)
    _check(lib().fp4_rope_table(_ptr(positions), T, axes, dims, theta, factor, window, amplitude, _ptr(table),
                                _stream(stream)), "fp4_rope_table")


def fp4_qk_norm_rope(q, q_stride: int, H_q: int, k, k_stride: int, H_k: int, T: int, D: int, norm, q_weight, k_weight,
                     eps: float, table, rot: int, layout, q_out, q_out_stride: int, k_out, k_out_stride: int,
                     stream=None):
    """q, k, q_out and k_out may be rows of a larger buffer (strides in elements)."""
    _check(lib().fp4_qk_norm_rope(_rows_ptr(q), q_stride, H_q, _rows_ptr(k), k_stride, H_k, T, D, _NORM[norm],
                                  _ptr(q_weight), _ptr(k_weight), eps, _ptr(table), rot, _ROPE[layout],
                                  _rows_ptr(q_out), q_out_stride, _rows_ptr(k_out), k_out_stride, _stream(stream)),
           "fp4_qk_norm_rope")


def fp4_qk_norm_rope_quantize_heads(fmt, q, q_stride: int, H_q: int, k, k_stride: int, H_k: int, T: int, D: int, norm,
                                    q_weight, k_weight, eps: float, table, rot: int, layout, g_q, g_k, q_codes, q_sf,
                                    k_codes, k_sf, stream=None):
    """q and k may be rows of a larger buffer (strides in elements)."""
    _check(lib().fp4_qk_norm_rope_quantize_heads(_fmt(fmt), _rows_ptr(q), q_stride, H_q, _rows_ptr(k), k_stride, H_k,
                                                 T, D, _NORM[norm], _ptr(q_weight), _ptr(k_weight), eps, _ptr(table),
                                                 rot, _ROPE[layout], _ptr(g_q), _ptr(g_k), _ptr(q_codes), _ptr(q_sf),
                                                 _ptr(k_codes), _ptr(k_sf), _stream(stream)),
           "fp4_qk_norm_rope_quantize_heads")


def fp4_dequantize_heads(fmt, codes, sf, T: int, H: int, D: int, g, x, x_stride: int, stream=None):
    """x may be rows of a larger buffer (x_stride in elements)."""
    _check(lib().fp4_dequantize_heads(_fmt(fmt), _ptr(codes), _ptr(sf), T, H, D, _ptr(g), _rows_ptr(x), x_stride,
                                      _stream(stream)), "fp4_dequantize_heads")


def fp4_attn_bf16_workspace_bytes(T_q: int, T_kv: int, H: int, H_kv: int, D: int = 128) -> int:
    return lib().fp4_attn_bf16_workspace_bytes(T_q, T_kv, H, H_kv, D)


def fp4_attn_bf16(q, q_stride: int, T_q: int, k, k_stride: int, v, v_stride: int, T_kv: int, H: int, H_kv: int, D: int,
                  scale: float, softcap: float, slopes, q_pos: int, key_start, key_end, o, o_stride: int, lse,
                  workspace, ws_bytes: int, stream=None):
    """q, k, v and o may be rows of larger buffers (strides in elements)."""
    _check(lib().fp4_attn_bf16(_rows_ptr(q), q_stride, T_q, _rows_ptr(k), k_stride, _rows_ptr(v), v_stride, T_kv, H,
                               H_kv, D, scale, softcap, _ptr(slopes), q_pos, _ptr(key_start), _ptr(key_end),
                               _rows_ptr(o), o_stride, _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)),
           "fp4_attn_bf16")


def fp4_attn_ranges(q_offsets, k_offsets, docs: int, T_q: int, T_kv: int, causal, prefix, key_start, key_end,
                    stream=None):
    _check(lib().fp4_attn_ranges(_ptr(q_offsets), _ptr(k_offsets), docs, T_q, T_kv, int(bool(causal)), _ptr(prefix),
                                 _ptr(key_start), _ptr(key_end), _stream(stream)), "fp4_attn_ranges")


def fp4_sync_status(stream=None) -> int:
    return lib().fp4_sync_status(_stream(stream))


def fp4_status_string(status: int) -> str:
    return lib().fp4_status_string(status).decode()


def fp4_set_wait_timeout_ns(ns: int):
    lib().fp4_set_wait_timeout_ns(ns)


def fp4bsa_clock_probe(out, blocks: int, stream=None):
    """Measurement hook: out (int64 [3 * blocks], device) = (SM id, SM cycle counter, global
    ns timer) per block, recorded by a tiny kernel on `stream`."""
    _check(lib().fp4bsa_clock_probe(_ptr(out), blocks, _stream(stream)), "fp4bsa_clock_probe")


def fp4bsa_test_gelu_f32(z, n: int, g, stream=None):
    """Test hook: g (fp32, device) = the library's fp32 GELU-tanh of each bf16 z (device),
    before the bf16 rounding the fused activation applies."""
    _check(lib().fp4bsa_test_gelu_f32(_ptr(z), n, _ptr(g), _stream(stream)), "fp4bsa_test_gelu_f32")


# ----------------------------------------------------------------------------- helpers
@dataclass
class PackedWeight:
    fmt: int
    N: int
    K: int
    codes: "object"          # torch.uint8 [N, K/2]
    sf: "object"             # torch.uint8 [sf bytes]
    w_global: "object" = None  # torch.float32 [1] (NVFP4)


def pack_weight(w, fmt="mxfp4", stream=None) -> PackedWeight:
    """bf16 [N, K] weight (CUDA) -> PackedWeight (codes, scales, NVFP4 global)."""
    import torch

    f = _fmt(fmt)
    N, K = w.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    sf = torch.empty(fp4_sf_bytes(f, N, K), dtype=torch.uint8, device=w.device)
    g = torch.empty(1, dtype=torch.float32, device=w.device) if f == NVFP4 else None
    fp4_pack_weight(f, w, N, K, codes, sf, g, stream)
    return PackedWeight(f, N, K, codes, sf, g)


def calibrate_act_global(batches, stream=None):
    """NVFP4 static activation global from one or more bf16 calibration batches (CUDA):
    returns (g_a, amax) as one-element fp32 device tensors."""
    import torch

    batches = [batches] if hasattr(batches, "is_cuda") else list(batches)
    dev = batches[0].device
    amax = torch.zeros(1, dtype=torch.float32, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    for b in batches:
        fp4_calibrate_act_global(b, b.numel(), amax, g, stream)
    return g, amax


def quantize_act(x, fmt="mxfp4", a_global=None, stream=None):
    """bf16 [M, K] activations (CUDA) -> (codes [M, K/2], scale factors)."""
    import torch

    f = _fmt(fmt)
    M, K = x.shape
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    sf = torch.empty(fp4_sf_bytes(f, M, K), dtype=torch.uint8, device=x.device)
    fp4_quantize_act(f, x, M, K, a_global, codes, sf, stream)
    return codes, sf


def quantize_heads(x, H: int, fmt="mxfp4", g=None, stream=None):
    """bf16 [T, H * 128] (CUDA) -> head-major (codes [H, Tpad, 64], scales [H, sf bytes per head])."""
    import torch

    f = _fmt(fmt)
    T, HD = x.shape
    D = HD // H
    Tpad = (T + 127) // 128 * 128
    codes = torch.empty((H, Tpad, D // 2), dtype=torch.uint8, device=x.device)
    sf = torch.empty((H, fp4_heads_sf_bytes(f, T, H, D) // H), dtype=torch.uint8, device=x.device)
    fp4_quantize_heads(f, x, T, H, D, g, codes, sf, stream)
    return codes, sf


def attn_scores(q_heads, k_heads, T_q: int, T_kv: int, head: int, fmt="mxfp4", g_q=None, g_k=None, s=None,
                stream=None):
    """Scores of one head from quantize_heads outputs: bf16 [T_q, T_kv rounded up to 128]."""
    import torch

    f = _fmt(fmt)
    qc, qs = q_heads
    kc, ks = k_heads
    H, _, half_d = qc.shape
    if s is None:
        s = torch.empty((T_q, (T_kv + 127) // 128 * 128), dtype=torch.bfloat16, device=qc.device)
    fp4_attn_scores(f, qc, qs, T_q, kc, ks, T_kv, H, 2 * half_d, head, g_q, g_k, s, stream)
    return s


P_GLOBAL_NVFP4 = 1.0 / 2688.0   # P's NVFP4 global: p <= 1, so T / (6 * 448) with T = 1


def quantize_heads_vt(v, H: int, fmt="mxfp4", g=None, stream=None):
    """bf16 [T, H * 128] (CUDA) -> head-major V^T (codes [H, 128, Tpad/2], scales [H, bytes per head])."""
    import torch

    f = _fmt(fmt)
    T, HD = v.shape
    D = HD // H
    Tpad = (T + 127) // 128 * 128
    codes = torch.empty((H, D, Tpad // 2), dtype=torch.uint8, device=v.device)
    sf = torch.empty((H, fp4_heads_vt_sf_bytes(f, T, H, D) // H), dtype=torch.uint8, device=v.device)
    fp4_quantize_heads_vt(f, v, T, H, D, g, codes, sf, stream)
    return codes, sf


def attn_softmax_quant(s, T_q: int, T_kv: int, scale: float, fmt="mxfp4", p_global=None, stream=None):
    """Scores bf16 [T_q, T_kv_pad] (CUDA) -> (P codes [T_q, T_kv_pad/2], P scales, (m, l) stats [T_q, 2]).
    NVFP4 needs p_global (a one-element fp32 device tensor, P_GLOBAL_NVFP4)."""
    import torch

    f = _fmt(fmt)
    kpad = s.shape[1]
    p_codes = torch.empty((T_q, kpad // 2), dtype=torch.uint8, device=s.device)
    p_sf = torch.empty(fp4_sf_bytes(f, T_q, kpad), dtype=torch.uint8, device=s.device)
    stats = torch.empty((T_q, 2), dtype=torch.float32, device=s.device)
    fp4_attn_softmax_quant(f, s, T_q, T_kv, scale, p_global, stats, p_codes, p_sf, stream)
    return p_codes, p_sf, stats


def attn_pv(p, vt_heads, T_q: int, T_kv: int, head: int, fmt="mxfp4", p_global=None, v_global=None, o=None,
            normalize=True, stream=None):
    """O -> bf16 [T_q, 128] from attn_softmax_quant's (codes, scales, stats) and quantize_heads_vt's V^T:
    deq(P~) deq(V_head), each row divided by its softmax sum unless normalize is False."""
    import torch

    f = _fmt(fmt)
    p_codes, p_sf = p[0], p[1]
    stats = p[2] if (normalize and len(p) > 2) else None
    vc, vs = vt_heads
    H, D, _ = vc.shape
    if o is None:
        o = torch.empty((T_q, D), dtype=torch.bfloat16, device=p_codes.device)
    fp4_attn_pv(f, p_codes, p_sf, p_global, T_q, T_kv, vc, vs, v_global, H, D, head, stats, o, stream)
    return o


def attn_fused(q_heads, k_heads, vt_heads, T_q: int, T_kv: int, head: int, scale: float, fmt="mxfp4", g_q=None,
               g_k=None, g_v=None, p_global=None, o=None, stats=None, trace_tile=None, stream=None):
    """One head's FP4 attention in one kernel (streaming form) from quantize_heads' Q and K and
    quantize_heads_vt's V^T: bf16 [T_q, 128].  NVFP4: the device fp32 globals of Q, K, V and P~
    (P_GLOBAL_NVFP4).  stats: an fp32 [T_q, 2] tensor to receive (final running maximum, l), or
    None.  trace_tile: a query tile whose per-block running maxima, P~ codes and scale bytes are
    returned too, as (o, (m [nblk, 128], codes [nblk, 128, 128], sf [nblk, 128, 256 / G]))."""
    import torch

    qc, qs = q_heads
    kc, ks = k_heads
    vc, vs = vt_heads
    H, _, half_d = qc.shape
    D = 2 * half_d
    if o is None:
        o = torch.empty((T_q, D), dtype=torch.bfloat16, device=qc.device)
    if trace_tile is None:
        fp4_attn_fused(fmt, qc, qs, T_q, kc, ks, T_kv, vc, vs, H, D, head, scale, g_q, g_k, g_v, p_global, stats, o,
                       stream)
        return o
    nblk = ((T_kv + 127) // 128 * 128 + 255) // 256
    G = 32 if _fmt(fmt) == MXFP4 else 16
    tm = torch.empty((nblk, 128), dtype=torch.float32, device=qc.device)
    tc = torch.empty((nblk, 128, 128), dtype=torch.uint8, device=qc.device)
    ts = torch.empty((nblk, 128, 256 // G), dtype=torch.uint8, device=qc.device)
    fp4_attn_fused_trace(fmt, qc, qs, T_q, kc, ks, T_kv, vc, vs, H, D, head, scale, g_q, g_k, g_v, p_global, stats, o,
                         trace_tile, tm, tc, ts, stream)
    return o, (tm, tc, ts)


def linear(x, pw: PackedWeight, bias=None, a_global=None, y=None, workspace=None, stream=None):
    """W4A4 quantized linear: bf16 [M, K] -> bf16 [M, N]."""
    import torch

    M, K = x.shape
    assert K == pw.K
    if y is None:
        y = torch.empty((M, pw.N), dtype=torch.bfloat16, device=x.device)
    ws = fp4_linear_workspace_bytes(pw.fmt, M, K, pw.N)
    if workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=x.device)
    fp4_linear(pw.fmt, x, M, K, pw.N, pw.codes, pw.sf, pw.w_global, a_global, bias, y, workspace,
               workspace.numel(), stream)
    return y


def w4a8_linear(x, r: PackedWeight, l1, l2, bias=None, y=None, workspace=None, stream=None):
    """W4A8 SVDQuant linear: bf16 [M, K] -> bf16 [M, N] (MXFP4 residual r, rank-32 L1 [K, rank]
    and L2 [rank, N] as stored)."""
    import torch

    M, K = x.shape
    rank = l1.shape[1]
    if y is None:
        y = torch.empty((M, r.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(w4a8_workspace_bytes(M, K, r.N, rank), dtype=torch.uint8, device=x.device)
    w4a8_svd_linear(x, M, K, r.N, r.codes, r.sf, l1, l2, rank, bias, y, workspace, workspace.numel(), stream)
    return y


def w4a4_linear(x, r: PackedWeight, l1, l2, bias=None, y=None, workspace=None, stream=None):
    """W4A4 SVDQuant linear: bf16 [M, K] -> bf16 [M, N] (MXFP4 activations and residual r,
    rank-32 L1 [K, rank] and L2 [rank, N] as stored)."""
    import torch

    M, K = x.shape
    rank = l1.shape[1]
    if y is None:
        y = torch.empty((M, r.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(w4a4_workspace_bytes(M, K, r.N, rank), dtype=torch.uint8, device=x.device)
    w4a4_svd_linear(x, M, K, r.N, r.codes, r.sf, l1, l2, rank, bias, y, workspace, workspace.numel(), stream)
    return y


def gelu_quantize_act(z, fmt="mxfp4", a_global=None, stream=None):
    """bf16 up-projection output z [M, K] (CUDA) -> (codes, scale factors) of
    bf16(gelu_tanh(z)) in fmt, the down projection's quantized input."""
    import torch

    f = _fmt(fmt)
    M, K = z.shape
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=z.device)
    sf = torch.empty(fp4_sf_bytes(f, M, K), dtype=torch.uint8, device=z.device)
    fp4_gelu_quantize_act(f, z, M, K, a_global, codes, sf, stream)
    return codes, sf


def linear_gelu_quant(x, pw: PackedWeight, bias=None, a_global=None, h_global=None, workspace=None, stream=None):
    """Up projection + GELU-tanh + quantize in one GEMM: bf16 x [M, K] -> (codes [M, N/2],
    scale factors) of h = bf16(gelu_tanh(bf16(x W^T + bias))) in the weight's format."""
    import torch

    M, K = x.shape
    N = pw.N
    codes = torch.empty((M, N // 2), dtype=torch.uint8, device=x.device)
    sf = torch.empty(fp4_sf_bytes(pw.fmt, M, N), dtype=torch.uint8, device=x.device)
    if workspace is None:
        workspace = torch.empty(fp4_linear_workspace_bytes(pw.fmt, M, K, N), dtype=torch.uint8, device=x.device)
    fp4_linear_gelu_quant(pw.fmt, x, M, K, N, pw.codes, pw.sf, pw.w_global, a_global, bias, h_global, codes, sf,
                          workspace, workspace.numel(), stream)
    return codes, sf


# ----------------------------------------------------------------------------- around the attention
# These helpers check types, shapes and devices, since the C calls see only addresses, and hand on
# addresses, so that nothing is checked twice: for small calls the host's time is what counts.
def _expect(t, what: str, dtype, dev: int, shape=None):
    """Address of t, which has to be a contiguous tensor of this type on CUDA device `dev` (and of this
    shape); None for None."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != dev or dev < 0:
        raise ValueError(f"{what}: expected {dtype} on cuda:{max(dev, 0)}, got {t.dtype} on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


def _expect_rows(t, what: str, dev: int, shape=None):
    """(address, row stride in elements) of t, which has to be a bf16 tensor [T, H, D] with contiguous heads on
    CUDA device `dev` (and of this shape)."""
    import torch

    if t.dim() != 3 or t.dtype != torch.bfloat16 or t.get_device() != dev or dev < 0:
        raise ValueError(f"{what}: expected a bf16 CUDA tensor [T, H, D] on cuda:{max(dev, 0)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    T, H, D = t.shape
    row, head, one = t.stride()
    if one != 1 or (H > 1 and head != D):
        raise ValueError(f"{what}: heads must be contiguous (strides {t.stride()})")
    return t.data_ptr(), row if T > 1 else H * D


def _rows_like(out, what: str, x, dev: int, stream):
    """(out, its address and row stride): `out` checked, or a new tensor like x [T, H, D] (rows next to one another)."""
    if out is not None:
        return out, *_expect_rows(out, what, dev, x.shape)
    import torch

    out = _new(dev, stream, lambda: torch.empty_like(x, memory_format=torch.contiguous_format))
    return out, out.data_ptr(), x.shape[1] * x.shape[2]


def _int64(value: int, what: str) -> int:
    """value, which has to fit the C call's 64 bits: ctypes cuts what does not, and the call would see another number."""
    if not -(1 << 63) <= value < 1 << 63:
        raise ValueError(f"{what}: {value} does not fit 64 bits")
    return value


def _launch(dev: int, call, *args):
    """The call with CUDA device `dev` current (its stream is that device's current one)."""
    import torch

    if torch.cuda.current_device() == dev:
        call(*args)
    else:
        with torch.cuda.device(dev):
            call(*args)


def _new(dev: int, stream, make):
    """make()'s tensor, allocated on `stream` where one is given: its memory may have been another
    tensor's of the current stream, and a workspace goes back to the allocator when the helper returns."""
    if stream is None:
        return make()
    import torch

    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return make()


def rope_table(positions, axis_dims, theta: float = 10000.0, factor: float = 1.0, window: int = 0,
               amplitude: float = 1.0, table=None, stream=None):
    """Rotary table of int32 positions [T, axes] (CUDA): fp32 [T, sum(axis_dims)] (cos, sin) pairs."""
    import torch

    if positions.dim() != 2 or positions.shape[1] != len(axis_dims):
        raise ValueError(f"positions: expected [T, {len(axis_dims)}], got {tuple(positions.shape)}")
    dev, T = positions.get_device(), positions.shape[0]
    pos = _expect(positions, "positions", torch.int32, dev)
    if table is None:
        table = _new(dev, stream, lambda: torch.empty((T, sum(axis_dims)), dtype=torch.float32, device=positions.device))
    _launch(dev, fp4_rope_table, pos, T, len(axis_dims), axis_dims, theta, factor, _int64(window, "window"), amplitude,
            _expect(table, "table", torch.float32, dev, (T, sum(axis_dims))), stream)
    return table


def _norm_rope_args(q, k, norm, q_weight, k_weight, eps, table, layout):
    """The leading arguments of both forms of fp4_qk_norm_rope, after checks."""
    import torch

    dev = q.get_device()
    qp, q_stride = _expect_rows(q, "q", dev)
    T, H_q, D = q.shape
    kp, k_stride, H_k = None, 0, 0
    if k is not None:
        kp, k_stride = _expect_rows(k, "k", dev)
        H_k = k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"k: expected [{T}, heads, {D}], got {tuple(k.shape)}")
    token = _NORM[norm] == NORM_TOKEN
    qw = _expect(q_weight, "q_weight", torch.float32, dev, (H_q * D if token else D,))
    kw = _expect(k_weight, "k_weight", torch.float32, dev, (H_k * D if token else D,))
    rot = 0 if table is None else table.shape[-1]
    tp = _expect(table, "table", torch.float32, dev, (T, rot))
    return qp, q_stride, H_q, kp, k_stride, H_k, T, D, norm, qw, kw, eps, tp, rot, layout


def qk_norm_rope(q, k=None, norm="head", q_weight=None, k_weight=None, eps: float = 1e-6, table=None,
                 layout="interleaved", q_out=None, k_out=None, stream=None):
    """RMS norm ("head", "token" or "none") and rotation of bf16 queries [T, H_q, D] and, if given, keys
    [T, H_k, D] in one launch; rows may be slices of a fused projection.  table: fp32 [T, rot] from
    rope_table, or None.  Returns (q_out, k_out), or q_out alone; q_out = q rotates in place."""
    args = _norm_rope_args(q, k, norm, q_weight, k_weight, eps, table, layout)
    dev = q.get_device()
    q_out, *outs = _rows_like(q_out, "q_out", q, dev, stream)
    if k is not None:
        k_out, *k_outs = _rows_like(k_out, "k_out", k, dev, stream)
        outs += k_outs
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        outs += [None, 0]
    _launch(dev, fp4_qk_norm_rope, *args, *outs, stream)
    return q_out if k is None else (q_out, k_out)


def qk_norm_rope_quantize_heads(q, k=None, fmt="mxfp4", norm="head", q_weight=None, k_weight=None, eps: float = 1e-6,
                                table=None, layout="interleaved", g_q=None, g_k=None, stream=None):
    """qk_norm_rope's result as head-major FP4 (codes, scales), as quantize_heads makes them of it:
    ((q_codes, q_sf), (k_codes, k_sf)), or the queries' pair alone.  NVFP4: g_q, g_k device globals."""
    import torch

    f = _fmt(fmt)
    args = _norm_rope_args(q, k, norm, q_weight, k_weight, eps, table, layout)
    dev, D = q.get_device(), q.shape[2]
    Tpad = (q.shape[0] + 127) // 128 * 128
    outs, ptrs = [], []
    for x in (q,) if k is None else (q, k):
        H = x.shape[1]
        if outs and H == q.shape[1]:  # (a tensor like another one is the quickest to have)
            codes, sf = (_new(dev, stream, lambda t=t: torch.empty_like(t)) for t in outs[0])
            outs.append((codes, sf))
            ptrs += [codes.data_ptr(), sf.data_ptr()]
            continue
        codes = _new(dev, stream, lambda: torch.empty((H, Tpad, D // 2), dtype=torch.uint8, device=q.device))
        sf = _new(dev, stream,
                  lambda: torch.empty((H, Tpad * (D // (32 if f == MXFP4 else 16))), dtype=torch.uint8, device=q.device))
        outs.append((codes, sf))
        ptrs += [codes.data_ptr(), sf.data_ptr()]
    if k is None:
        ptrs += [None, None]
    _launch(dev, fp4_qk_norm_rope_quantize_heads, f, *args, _expect(g_q, "g_q", torch.float32, dev),
            _expect(g_k, "g_k", torch.float32, dev), *ptrs, stream)
    return outs[0] if k is None else tuple(outs)


def dequantize_heads(heads, T: int, fmt="mxfp4", g=None, x=None, stream=None):
    """quantize_heads' (codes, scales) of T tokens back to bf16 [T, H, 128]."""
    import torch

    f = _fmt(fmt)
    codes, sf = heads
    dev = codes.get_device()
    H, Tpad, half_d = codes.shape
    if Tpad != (T + 127) // 128 * 128:
        raise ValueError(f"codes of {Tpad} padded tokens do not belong to {T} tokens")
    cp = _expect(codes, "codes", torch.uint8, dev)
    sp = _expect(sf, "scales", torch.uint8, dev, (H, Tpad * (2 * half_d // (32 if f == MXFP4 else 16))))
    if x is None:
        x = _new(dev, stream, lambda: torch.empty((T, H, 2 * half_d), dtype=torch.bfloat16, device=codes.device))
    _launch(dev, fp4_dequantize_heads, f, cp, sp, T, H, 2 * half_d, _expect(g, "g", torch.float32, dev),
            *_expect_rows(x, "x", dev, (T, H, 2 * half_d)), stream)
    return x


def linear_residual(x, pw: PackedWeight, residual=None, bias=None, act="none", gate=None, gate_rows: int = 0,
                    a_global=None, y=None, workspace=None, stream=None):
    """residual + gate * act(x W^T + bias) in the GEMM's epilogue: bf16 [M, K] -> bf16 [M, N].  gate: fp32
    [ceil(M / gate_rows), N], each row for gate_rows rows of y.  y = residual updates it in place."""
    import torch

    M, K = x.shape
    N, dev = pw.N, x.get_device()
    if K != pw.K:
        raise ValueError(f"x: expected [M, {pw.K}], got {tuple(x.shape)}")
    if gate is None:
        gate_rows = 0
    elif gate_rows < 1:
        raise ValueError("gate_rows: the number of rows of y that share a row of the gate")
    xp = _expect(x, "x", torch.bfloat16, dev)
    rp = _expect(residual, "residual", torch.bfloat16, dev, (M, N))
    bp = _expect(bias, "bias", torch.float16, dev, (N,))
    wp = _expect(pw.codes, "weight codes", torch.uint8, dev, (N, K // 2))
    wsp, wgp = _expect(pw.sf, "weight scales", torch.uint8, dev), _expect(pw.w_global, "w_global", torch.float32, dev)
    if pw.sf.numel() != fp4_sf_bytes(pw.fmt, N, K):
        raise ValueError(f"weight scales: expected {fp4_sf_bytes(pw.fmt, N, K)} bytes, got {pw.sf.numel()}")
    gate_rows = min(gate_rows, max(M, 1))
    gp = None if gate is None else _expect(gate, "gate", torch.float32, dev, (-(-M // gate_rows), N))
    if y is None:
        y = _new(dev, stream, lambda: torch.empty((M, N), dtype=torch.bfloat16, device=x.device))
    if workspace is None:
        size = fp4_linear_workspace_bytes(pw.fmt, M, K, N)
        workspace = _new(dev, stream, lambda: torch.empty(size, dtype=torch.uint8, device=x.device))
    _launch(dev, fp4_linear_residual, pw.fmt, xp, M, K, N, wp, wsp, wgp,
            _expect(a_global, "a_global", torch.float32, dev), bp, act, gp, gate_rows, rp,
            _expect(y, "y", torch.bfloat16, dev, (M, N)), _expect(workspace, "workspace", torch.uint8, dev),
            workspace.numel(), stream)
    return y


def attn_ranges(q_offsets, k_offsets, T_q: int, T_kv: int, causal=False, prefix=None, stream=None):
    """Key ranges (key_start, key_end), int32 [T_q], of documents packed on the query and key axes (int32
    offsets [docs + 1], CUDA), in causal order or not, each with a prefix (int32 [docs]) that all its rows see."""
    import torch

    dev, docs = q_offsets.get_device(), q_offsets.numel() - 1
    qp = _expect(q_offsets, "q_offsets", torch.int32, dev, (docs + 1,))
    kp = _expect(k_offsets, "k_offsets", torch.int32, dev, (docs + 1,))
    pp = _expect(prefix, "prefix", torch.int32, dev, (docs,))
    _int64(T_kv, "T_kv")
    start, end = (_new(dev, stream, lambda: q_offsets.new_empty(T_q)) for _ in range(2))
    _launch(dev, fp4_attn_ranges, qp, kp, docs, T_q, T_kv, causal, pp, start.data_ptr(), end.data_ptr(), stream)
    return start, end


def attn_bf16(q, k, v, scale: float, softcap: float = 0.0, slopes=None, q_pos: int = 0, key_start=None, key_end=None,
              o=None, return_lse=False, workspace=None, stream=None):
    """Attention of bf16 q [T_q, H, D] over k, v [T_kv, H_kv, D] (slices of fused projections do): bf16
    [T_q, H, D], and with return_lse its fp32 log-sum-exp [T_q, H].  softcap > 0 caps the scores by a tanh,
    slopes (fp32 [H]) times the distance |q_pos + i - j| is taken from them, and row i sees the keys
    key_start[i] <= j < key_end[i] (int32 [T_q]; None: from the first, to the last)."""
    import torch

    dev = q.get_device()
    qp, q_stride = _expect_rows(q, "q", dev)
    T_q, H, D = q.shape
    kp, k_stride = _expect_rows(k, "k", dev)
    T_kv, H_kv, _ = k.shape
    if k.shape[2] != D:
        raise ValueError(f"k: expected [T_kv, H_kv, {D}], got {tuple(k.shape)}")
    vp, v_stride = _expect_rows(v, "v", dev, k.shape)
    o, op, o_stride = _rows_like(o, "o", q, dev, stream)
    lse = None
    if return_lse:
        lse = _new(dev, stream, lambda: torch.empty((T_q, H), dtype=torch.float32, device=q.device))
    ws = fp4_attn_bf16_workspace_bytes(T_q, T_kv, H, H_kv, D)
    if workspace is None and ws:
        workspace = _new(dev, stream, lambda: torch.empty(ws, dtype=torch.uint8, device=q.device))
    wp = _expect(workspace, "workspace", torch.uint8, dev)
    _launch(dev, fp4_attn_bf16, qp, q_stride, T_q, kp, k_stride, vp, v_stride, T_kv, H, H_kv, D, scale, softcap,
            _expect(slopes, "slopes", torch.float32, dev, (H,)), _int64(q_pos, "q_pos"),
            _expect(key_start, "key_start", torch.int32, dev, (T_q,)),
            _expect(key_end, "key_end", torch.int32, dev, (T_q,)), op, o_stride,
            None if lse is None else lse.data_ptr(), wp, 0 if workspace is None else workspace.numel(), stream)
    return (o, lse) if return_lse else o


class HostPipeline:
    """Reusable device buffers, streams and events for linear_host: two sets of per-chunk
    device buffers (x rows, y rows, quantize workspace) so that the host->device copy of
    chunk i + 1, the linear of chunk i and the device->host copy of chunk i - 1 run
    concurrently on three streams."""

    def __init__(self, fmt, chunk_rows: int, K: int, N: int, device="cuda"):
        import torch

        self.fmt = _fmt(fmt)
        self.chunk_rows, self.K, self.N = chunk_rows, K, N
        ws = fp4_linear_workspace_bytes(self.fmt, chunk_rows, K, N)
        self.x = [torch.empty((chunk_rows, K), dtype=torch.bfloat16, device=device) for _ in range(2)]
        self.y = [torch.empty((chunk_rows, N), dtype=torch.bfloat16, device=device) for _ in range(2)]
        self.ws = [torch.empty(ws, dtype=torch.uint8, device=device) for _ in range(2)]
        self.streams = [torch.cuda.Stream(device=device) for _ in range(3)]
        self.ev_x = [torch.cuda.Event() for _ in range(2)]   # chunk copied in
        self.ev_c = [torch.cuda.Event() for _ in range(2)]   # chunk computed (x read, y written)
        self.ev_y = [torch.cuda.Event() for _ in range(2)]   # chunk copied out


def linear_host(x_host, pw: PackedWeight, pipe: HostPipeline, bias=None, a_global=None, y_host=None):
    """Host-to-host W4A4 linear: pinned bf16 x [M, K] in host memory -> pinned bf16 y
    [M, N] in host memory, in row chunks of pipe.chunk_rows through fp4_linear, with the
    copies in both directions overlapped with the GEMMs (see HostPipeline).  The work is
    ordered after everything already on the current stream, and the current stream waits
    for the last copy, so an event recorded on it afterwards marks completion."""
    import torch

    M, K = x_host.shape
    assert K == pipe.K and pw.N == pipe.N and pw.fmt == pipe.fmt
    if y_host is None:
        y_host = torch.empty((M, pw.N), dtype=torch.bfloat16, pin_memory=True)
    cur = torch.cuda.current_stream()
    s_in, s_mm, s_out = pipe.streams
    for s in pipe.streams:
        s.wait_stream(cur)
    C = pipe.chunk_rows
    for i, r0 in enumerate(range(0, M, C)):
        r1 = min(M, r0 + C)
        rows, b = r1 - r0, i % 2
        xd, yd = pipe.x[b][:rows], pipe.y[b][:rows]
        with torch.cuda.stream(s_in):
            if i >= 2:
                s_in.wait_event(pipe.ev_c[b])        # chunk i - 2 no longer reads x[b]
            xd.copy_(x_host[r0:r1], non_blocking=True)
            pipe.ev_x[b].record(s_in)
        with torch.cuda.stream(s_mm):
            s_mm.wait_event(pipe.ev_x[b])
            if i >= 2:
                s_mm.wait_event(pipe.ev_y[b])        # chunk i - 2 copied y[b] out
            fp4_linear(pipe.fmt, xd, rows, K, pipe.N, pw.codes, pw.sf, pw.w_global, a_global, bias, yd,
                       pipe.ws[b], pipe.ws[b].numel(), s_mm)
            pipe.ev_c[b].record(s_mm)
        with torch.cuda.stream(s_out):
            s_out.wait_event(pipe.ev_c[b])
            y_host[r0:r1].copy_(yd, non_blocking=True)
            pipe.ev_y[b].record(s_out)
    cur.wait_stream(s_out)
    return y_host
