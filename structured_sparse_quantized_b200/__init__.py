"""structured_sparse_quantized_b200 -- Python binding of libss.

Quantized (INT8 / FP8-E4M3, and the unscaled BF16 tier) matmul on the
Blackwell sparse tensor cores for
structured-sparse weights: hardware 2:4 and the milder (2Nh-2):2Nh patterns
(4:6, 6:8, 8:10) brought to 2:4 by SlideSparse's sliding-window
decomposition.  Every step runs in the CUDA kernels of ``libss.so`` (see
``include/ss.h``); this module only marshals arguments: torch tensors supply
device memory and streams, and each ``ss_*`` function here calls the C
function of the same name.  There is no CPU fallback: if ``libss.so`` is
missing, or the device is not sm_100, calls raise ``SSError``.

Low-level calls (same names and argument order as the C ABI, outputs
preallocated by the caller):
    ss_parse_pattern, ss_slide_shape, ss_act_2to4_shape, ss_compress_weight,
    ss_quant_lift_act, ss_prune_act_2to4, ss_sparse_gemm, ss_dense_gemm,
    ss_get_device_status, ss_status_string, ss_kernel_launches, ss_meta_bytes,
    ss_debug_set_wait_limit, ss_debug_skip_stage (test hooks),
    ss_fp4_shape, ss_fp4_scale_bytes, ss_compress_weight_nvfp4,
    ss_quant_lift_act_nvfp4, ss_sparse_gemm_nvfp4, ss_dense_gemm_nvfp4,
    ss_sparse_gemm_fused, ss_dense_gemm_fused, ss_sparse_gemm_nvfp4_fused,
    ss_dense_gemm_nvfp4_fused (bias, activation, residual: Epilogue),
    ss_norm_quant_lift_act, ss_rope, ss_rope_frequencies
Convenience wrappers that allocate their outputs with torch:
    compress_weight, quant_lift_act, prune_act_2to4, sparse_gemm, dense_gemm,
    linear, and for NVFP4 compress_weight_nvfp4, quant_lift_act_nvfp4,
    sparse_gemm_nvfp4, dense_gemm_nvfp4, linear_nvfp4; the GEMMs and linears
    take an optional epilogue=Epilogue(...).
    norm_quant_lift_act, rope, rope_frequencies, interleave_gate_up, and the
    two halves of a transformer layer around its attention: project_qkv
    (norm, product, rotary positions), feed_forward (norm, gated product,
    product into the residual stream).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libss.so")

SS_OK = 0
SS_ERR_INVALID_ARG = 1
SS_ERR_UNSUPPORTED = 2
SS_ERR_ALIGNMENT = 3
SS_ERR_ARCH = 4
SS_ERR_CUDA = 5
SS_ERR_TIMEOUT = 6
SS_ERR_DATA = 7

SS_IN_F32, SS_IN_BF16 = 0, 1
SS_INT8, SS_FP8_E4M3, SS_BF16 = 0, 1, 2
SS_OUT_F32, SS_OUT_BF16 = 0, 1

SS_ACT_NONE, SS_ACT_RELU, SS_ACT_SILU, SS_ACT_GELU, SS_ACT_GELU_ERF = 0, 1, 2, 3, 4
SS_ROPE_HALF, SS_ROPE_INTERLEAVED = 0, 1
SS_ROPE_NONE, SS_ROPE_LINEAR, SS_ROPE_NTK, SS_ROPE_LLAMA3, SS_ROPE_YARN = 0, 1, 2, 3, 4

ACTS = {"none": SS_ACT_NONE, "relu": SS_ACT_RELU, "silu": SS_ACT_SILU, "gelu": SS_ACT_GELU,
        "gelu_erf": SS_ACT_GELU_ERF}
ROPE_LAYOUTS = {"half": SS_ROPE_HALF, "interleaved": SS_ROPE_INTERLEAVED}
ROPE_KINDS = {"none": SS_ROPE_NONE, "linear": SS_ROPE_LINEAR, "ntk": SS_ROPE_NTK,
              "llama3": SS_ROPE_LLAMA3, "yarn": SS_ROPE_YARN}
QDTYPES = {"int8": SS_INT8, "fp8": SS_FP8_E4M3, "e4m3": SS_FP8_E4M3, "bf16": SS_BF16}


class SSError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {ss_status_string(status)} ({status})")
        self.status = status


class ss_pattern(ctypes.Structure):
    _fields_ = [("keep", ctypes.c_int32), ("group", ctypes.c_int32)]


class ss_epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("bias_dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("gated", ctypes.c_int32)]


class ss_rope_heads(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("in_token", ctypes.c_int64), ("in_head", ctypes.c_int64),
                ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64)]


class ss_rope_scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double),
                ("original", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libss.so (built by ``python -m structured_sparse_quantized_b200._build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libss.so is not built ({LIB_PATH}); run "
                           "`python -m structured_sparse_quantized_b200._build`")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, p, f = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
    pat = ss_pattern
    sigs = {
        "ss_parse_pattern": [ctypes.c_char_p, ctypes.POINTER(pat)],
        "ss_slide_shape": [pat, i64, ctypes.POINTER(i64), ctypes.POINTER(i64),
                           ctypes.POINTER(i64)],
        "ss_act_2to4_shape": [i64, ctypes.POINTER(i64)],
        "ss_compress_weight": [p, i32, i64, i64, pat, i32, p, p, p, p],
        "ss_quant_lift_act": [p, i32, i64, i64, pat, i32, p, p, p],
        "ss_prune_act_2to4": [p, i32, i64, i64, i32, p, p, p, p],
        "ss_sparse_gemm": [i32, p, p, p, p, p, i64, i64, i64, i32, p, i32, p],
        "ss_dense_gemm": [p, p, p, p, i64, i64, i64, i32, p, i32, p],
        "ss_get_device_status": [p],
        "ss_debug_set_wait_limit": [ctypes.c_uint64],
        "ss_debug_skip_stage": [i32],
        "ss_fp4_shape": [pat, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)],
        "ss_compress_weight_nvfp4": [p, i32, i64, i64, pat, p, p, p, p, p],
        "ss_quant_lift_act_nvfp4": [p, i32, i64, i64, pat, i32, p, p, p, p],
        "ss_sparse_gemm_nvfp4": [p, p, p, p, p, p, p, i64, i64, i64, p, i32, p],
        "ss_dense_gemm_nvfp4": [p, p, p, p, p, p, i64, i64, i64, p, i32, p],
        "ss_sparse_gemm_fused": [i32, p, p, p, p, p, i64, i64, i64, i32, p, p, i32, p],
        "ss_dense_gemm_fused": [p, p, p, p, i64, i64, i64, i32, p, p, i32, p],
        "ss_sparse_gemm_nvfp4_fused": [p, p, p, p, p, p, p, i64, i64, i64, p, p, i32, p],
        "ss_dense_gemm_nvfp4_fused": [p, p, p, p, p, p, i64, i64, i64, p, p, i32, p],
        "ss_norm_quant_lift_act": [p, i32, p, i32, f, i64, i64, pat, i32, p, p, p],
        "ss_rope": [p, p, i32, p, ctypes.c_int32, p, f, i64, i64, i64, i32, p],
        "ss_rope_frequencies": [i64, ctypes.c_double, p, p, p],
    }
    for name, args in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = i32
    L.ss_status_string.argtypes = [i32]
    L.ss_status_string.restype = ctypes.c_char_p
    L.ss_kernel_launches.argtypes = []
    L.ss_kernel_launches.restype = i64
    L.ss_meta_bytes.argtypes = [i64, i64]
    L.ss_meta_bytes.restype = i64
    L.ss_fp4_scale_bytes.argtypes = [i64, i64, i32]
    L.ss_fp4_scale_bytes.restype = i64
    _lib = L
    return L


def ss_status_string(status: int) -> str:
    return lib().ss_status_string(int(status)).decode()


def ss_kernel_launches() -> int:
    return int(lib().ss_kernel_launches())


def _check(status: int, where: str) -> None:
    if status != SS_OK:
        raise SSError(status, where)


# ------------------------------------------------------------------ marshalling

def _pattern(p) -> ss_pattern:
    if isinstance(p, ss_pattern):
        return p
    out = ss_pattern()
    _check(lib().ss_parse_pattern(str(p).encode(), ctypes.byref(out)), "ss_parse_pattern")
    return out


def _qdtype(q) -> int:
    return QDTYPES[q] if isinstance(q, str) else int(q)


def _dev(t: torch.Tensor | None, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _in_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SS_IN_BF16
    if t.dtype == torch.float32:
        return SS_IN_F32
    raise ValueError(f"input dtype {t.dtype} not supported (float32 or bfloat16)")


def _out_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SS_OUT_BF16
    if t.dtype == torch.float32:
        return SS_OUT_F32
    raise ValueError(f"output dtype {t.dtype} not supported (float32 or bfloat16)")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


# ------------------------------------------------------------------ C ABI, 1:1

def ss_parse_pattern(s: str) -> tuple[int, int]:
    p = _pattern(s)
    return p.keep, p.group


def ss_slide_shape(pattern, K: int) -> tuple[int, int, int]:
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().ss_slide_shape(_pattern(pattern), int(K), ctypes.byref(a), ctypes.byref(b),
                                ctypes.byref(c)), "ss_slide_shape")
    return a.value, b.value, c.value


def ss_act_2to4_shape(K: int) -> int:
    a = ctypes.c_int64()
    _check(lib().ss_act_2to4_shape(int(K), ctypes.byref(a)), "ss_act_2to4_shape")
    return a.value


def ss_meta_bytes(rows: int, K_lp: int) -> int:
    return int(lib().ss_meta_bytes(int(rows), int(K_lp)))


def meta_shape(rows: int, K_lp: int) -> tuple:
    """Shape of a tile-major metadata buffer: [row tiles, K tiles, 128, 16]
    (one 2 KB block of 2:4 selectors per 128 rows x 128 lifted K)."""
    return ((rows + 127) // 128, K_lp // 128, 128, 16)


def ss_compress_weight(W, pattern, q, Wv, Wm, s_w, stream=None) -> None:
    N, K = W.shape
    _check(lib().ss_compress_weight(_dev(W, "W"), _in_dtype(W), N, K, _pattern(pattern),
                                    _qdtype(q), _dev(Wv, "Wv"), _dev(Wm, "Wm"),
                                    _dev(s_w, "s_w"), _stream(stream)), "ss_compress_weight")


def ss_quant_lift_act(X, pattern, q, Xq_lift, s_x, stream=None) -> None:
    M, K = X.shape
    _check(lib().ss_quant_lift_act(_dev(X, "X"), _in_dtype(X), M, K, _pattern(pattern),
                                   _qdtype(q), _dev(Xq_lift, "Xq_lift"), _dev(s_x, "s_x"),
                                   _stream(stream)), "ss_quant_lift_act")


def ss_prune_act_2to4(X, q, Xv, Xm, s_x, stream=None) -> None:
    M, K = X.shape
    _check(lib().ss_prune_act_2to4(_dev(X, "X"), _in_dtype(X), M, K, _qdtype(q),
                                   _dev(Xv, "Xv"), _dev(Xm, "Xm"), _dev(s_x, "s_x"),
                                   _stream(stream)), "ss_prune_act_2to4")


def ss_sparse_gemm(sparse_operand: int, Av, Am, s_a, B, s_b, M: int, N: int, K_lp: int, q, Y,
                   stream=None) -> None:
    _check(lib().ss_sparse_gemm(int(sparse_operand), _dev(Av, "Av"), _dev(Am, "Am"),
                                _dev(s_a, "s_a"), _dev(B, "B"), _dev(s_b, "s_b"), int(M), int(N),
                                int(K_lp), _qdtype(q), _dev(Y, "Y"), _out_dtype(Y),
                                _stream(stream)), "ss_sparse_gemm")


def ss_dense_gemm(Xq, s_x, Wq, s_w, M: int, N: int, K_p: int, q, Y, stream=None) -> None:
    _check(lib().ss_dense_gemm(_dev(Xq, "Xq"), _dev(s_x, "s_x"), _dev(Wq, "Wq"),
                               _dev(s_w, "s_w"), int(M), int(N), int(K_p), _qdtype(q),
                               _dev(Y, "Y"), _out_dtype(Y), _stream(stream)), "ss_dense_gemm")


def ss_get_device_status(stream=None) -> int:
    return int(lib().ss_get_device_status(_stream(stream)))


def ss_debug_set_wait_limit(ns: int) -> None:
    """Test hook: device-side waits give up after `ns` nanoseconds (4 s default)."""
    _check(lib().ss_debug_set_wait_limit(int(ns)), "ss_debug_set_wait_limit")


def ss_debug_skip_stage(kb: int) -> None:
    """Test hook: GEMM producers skip K stage `kb` of their first tile (-1: off)."""
    _check(lib().ss_debug_skip_stage(int(kb)), "ss_debug_skip_stage")


# ------------------------------------------------------------------ allocating wrappers
# Stored values are uint8 codes for the 8-bit tiers and bfloat16 for the bf16
# tier, which has no scales (its s_* entries are None).  What a call allocates,
# outputs and intermediates, is allocated for the stream that it runs on.

def _vals_dtype(q) -> torch.dtype:
    return torch.bfloat16 if _qdtype(q) == SS_BF16 else torch.uint8


def _new(like: torch.Tensor, shape, dtype, stream):
    """A tensor on like's device, allocated for the stream that will write it (so
    that its memory is reused in that stream's order)."""
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    with _as_current(stream, like):
        return like.new_empty(shape, dtype=dtype)


def _as_current(stream, like: torch.Tensor):
    """Context in which `stream` (a Stream or a handle) is the current one."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    return torch.cuda.stream(stream)


def _away(X: torch.Tensor, stream):
    """Context in which `stream`, or else X's device, is the current one; None
    where it is already."""
    d = _index(X, "X")
    if stream is not None:
        return _as_current(stream, X)
    return None if torch._C._cuda_getDevice() == d else torch.cuda.device(d)


def _scales(like: torch.Tensor, n: int, q, stream):
    return None if _qdtype(q) == SS_BF16 else _new(like, (n,), torch.float32, stream)


def compress_weight(W: torch.Tensor, pattern, q, stream=None):
    """-> (Wv, Wm, s_w); Wm is None for 'dense'."""
    N, K = W.shape
    p = _pattern(pattern)
    _, _, K_lp = ss_slide_shape(p, K)
    vd = _vals_dtype(q)
    if p.group == 0:
        Wv = _new(W, (N, K_lp), vd, stream)
        Wm = None
    else:
        Wv = _new(W, (N, K_lp // 2), vd, stream)
        Wm = _new(W, meta_shape(N, K_lp), torch.uint8, stream)
    s_w = _scales(W, N, q, stream)
    ss_compress_weight(W, p, q, Wv, Wm, s_w, stream)
    return Wv, Wm, s_w


def quant_lift_act(X: torch.Tensor, pattern, q, stream=None, out=None):
    M, K = X.shape
    p = _pattern(pattern)
    _, _, K_lp = ss_slide_shape(p, K)
    if out is None:
        out = (_new(X, (M, K_lp), _vals_dtype(q), stream), _scales(X, M, q, stream))
    ss_quant_lift_act(X, p, q, out[0], out[1], stream)
    return out


def prune_act_2to4(X: torch.Tensor, q, stream=None, out=None):
    M, K = X.shape
    K_lp = ss_act_2to4_shape(K)
    if out is None:
        out = (_new(X, (M, K_lp // 2), _vals_dtype(q), stream),
               _new(X, meta_shape(M, K_lp), torch.uint8, stream), _scales(X, M, q, stream))
    ss_prune_act_2to4(X, q, out[0], out[1], out[2], stream)
    return out


def sparse_gemm(sparse_operand: int, Av, Am, s_a, B, s_b, M: int, N: int, q,
                out_dtype=torch.bfloat16, stream=None, out=None, epilogue=None):
    K_lp = Av.shape[1] * 2
    if epilogue is not None:
        out = epilogue._out(M, N, out_dtype, Av, out, stream)
        ss_sparse_gemm_fused(sparse_operand, Av, Am, s_a, B, s_b, M, N, K_lp, q, epilogue, out,
                             stream)
        return out
    if out is None:
        out = _new(Av, (M, N), out_dtype, stream)
    ss_sparse_gemm(sparse_operand, Av, Am, s_a, B, s_b, M, N, K_lp, q, out, stream)
    return out


def dense_gemm(Xq, s_x, Wq, s_w, q, out_dtype=torch.bfloat16, stream=None, out=None,
               epilogue=None):
    M, K_p = Xq.shape
    N = Wq.shape[0]
    if epilogue is not None:
        out = epilogue._out(M, N, out_dtype, Xq, out, stream)
        ss_dense_gemm_fused(Xq, s_x, Wq, s_w, M, N, K_p, q, epilogue, out, stream)
        return out
    if out is None:
        out = _new(Xq, (M, N), out_dtype, stream)
    ss_dense_gemm(Xq, s_x, Wq, s_w, M, N, K_p, q, out, stream)
    return out


def linear(X: torch.Tensor, packed, pattern, q, out_dtype=torch.bfloat16, stream=None,
           epilogue=None, norm=None, out=None):
    """Y = X W^T through the weight-sparse path: quant+lift, then the sparse
    GEMM (or the dense GEMM for pattern 'dense').  `packed` = compress_weight().
    norm = (weight, eps): RMS norm of X fused into the quantisation.
    epilogue: bias, activation and residual fused into the GEMM.
    out: the [M, N] output (a gated one [M, N/2])."""
    away = _away(X, stream)
    if away is not None:
        with away:  # the quantised activation is that stream's too
            return linear(X, packed, pattern, q, out_dtype, None, epilogue, norm, out)
    Wv, Wm, s_w = packed
    M, K = X.shape
    N = Wv.shape[0]
    p, K_lp = _pattern_k_lp(pattern, K)
    _fits(M, N, K, K_lp, Wv.shape[1] * (1 if p.group == 0 else 2), out, epilogue)
    if norm is None:
        Xq, s_x = quant_lift_act(X, pattern, q, stream)
    else:
        Xq, s_x = norm_quant_lift_act(X, norm[0], norm[1], pattern, q, stream)
    if p.group == 0:
        return dense_gemm(Xq, s_x, Wv, s_w, q, out_dtype, stream, out, epilogue)
    return sparse_gemm(0, Wv, Wm, s_w, Xq, s_x, M, N, q, out_dtype, stream, out, epilogue)


# ------------------------------------------------------------------ NVFP4 (pairwise sparse FP4)
# Patterns count pairs of adjacent elements ("2:4" = the hardware's pairwise
# 4:8).  Values are packed E2M1 codes (uint8, two per byte), local scales
# UE4M3 bytes in the tile-major layout of ss_fp4_scale_bytes, global scales
# fp32 (one per weight tensor, one per token).

def ss_fp4_shape(pattern, K: int) -> tuple[int, int]:
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().ss_fp4_shape(_pattern(pattern), int(K), ctypes.byref(a), ctypes.byref(b)),
           "ss_fp4_shape")
    return a.value, b.value


def ss_fp4_scale_bytes(rows: int, K_lp: int, block: int) -> int:
    return int(lib().ss_fp4_scale_bytes(int(rows), int(K_lp), int(block)))


def ss_compress_weight_nvfp4(W, pattern, Wv, Wm, Ws, g_w, stream=None) -> None:
    N, K = W.shape
    _check(lib().ss_compress_weight_nvfp4(_dev(W, "W"), _in_dtype(W), N, K, _pattern(pattern),
                                          _dev(Wv, "Wv"), _dev(Wm, "Wm"), _dev(Ws, "Ws"),
                                          _dev(g_w, "g_w"), _stream(stream)),
           "ss_compress_weight_nvfp4")


def ss_quant_lift_act_nvfp4(X, pattern, block: int, Xv, Xs, g_x, stream=None) -> None:
    M, K = X.shape
    _check(lib().ss_quant_lift_act_nvfp4(_dev(X, "X"), _in_dtype(X), M, K, _pattern(pattern),
                                         int(block), _dev(Xv, "Xv"), _dev(Xs, "Xs"),
                                         _dev(g_x, "g_x"), _stream(stream)),
           "ss_quant_lift_act_nvfp4")


def ss_sparse_gemm_nvfp4(Wv, Wm, Ws, g_w, Xv, Xs, g_x, M: int, N: int, K_lp: int, Y,
                         stream=None) -> None:
    _check(lib().ss_sparse_gemm_nvfp4(_dev(Wv, "Wv"), _dev(Wm, "Wm"), _dev(Ws, "Ws"),
                                      _dev(g_w, "g_w"), _dev(Xv, "Xv"), _dev(Xs, "Xs"),
                                      _dev(g_x, "g_x"), int(M), int(N), int(K_lp), _dev(Y, "Y"),
                                      _out_dtype(Y), _stream(stream)), "ss_sparse_gemm_nvfp4")


def ss_dense_gemm_nvfp4(Xv, Xs, g_x, Wv, Ws, g_w, M: int, N: int, K_p: int, Y,
                        stream=None) -> None:
    _check(lib().ss_dense_gemm_nvfp4(_dev(Xv, "Xv"), _dev(Xs, "Xs"), _dev(g_x, "g_x"),
                                     _dev(Wv, "Wv"), _dev(Ws, "Ws"), _dev(g_w, "g_w"), int(M),
                                     int(N), int(K_p), _dev(Y, "Y"), _out_dtype(Y),
                                     _stream(stream)), "ss_dense_gemm_nvfp4")


def compress_weight_nvfp4(W: torch.Tensor, pattern, stream=None):
    """-> (Wv, Wm, Ws, g_w); Wm is None for 'dense' (blocks of 16)."""
    N, K = W.shape
    p = _pattern(pattern)
    _, K_lp = ss_fp4_shape(p, K)
    if p.group == 0:
        Wv = _new(W, (N, K_lp // 2), torch.uint8, stream)
        Wm = None
        Ws = _new(W, (ss_fp4_scale_bytes(N, K_lp, 16),), torch.uint8, stream)
    else:
        Wv = _new(W, (N, K_lp // 4), torch.uint8, stream)
        Wm = _new(W, meta_shape(N, K_lp // 2), torch.uint8, stream)
        Ws = _new(W, (ss_fp4_scale_bytes(N, K_lp, 32),), torch.uint8, stream)
    g_w = _new(W, (4,), torch.float32, stream)   # [0] is the global scale
    ss_compress_weight_nvfp4(W, p, Wv, Wm, Ws, g_w, stream)
    return Wv, Wm, Ws, g_w


def quant_lift_act_nvfp4(X: torch.Tensor, pattern, block: int, stream=None, out=None):
    """-> (Xv [M, K_lp/2] uint8, Xs scale bytes, g_x: [0] is the tensor's global scale)."""
    M, K = X.shape
    p = _pattern(pattern)
    _, K_lp = ss_fp4_shape(p, K)
    if out is None:
        out = (_new(X, (M, K_lp // 2), torch.uint8, stream),
               _new(X, (ss_fp4_scale_bytes(M, K_lp, block),), torch.uint8, stream),
               _new(X, (4,), torch.float32, stream))
    ss_quant_lift_act_nvfp4(X, p, block, out[0], out[1], out[2], stream)
    return out


def sparse_gemm_nvfp4(packed, act, M: int, N: int, out_dtype=torch.bfloat16, stream=None,
                      out=None, epilogue=None):
    Wv, Wm, Ws, g_w = packed
    Xv, Xs, g_x = act
    K_lp = Xv.shape[1] * 2
    if epilogue is not None:
        out = epilogue._out(M, N, out_dtype, Xv, out, stream)
        ss_sparse_gemm_nvfp4_fused(Wv, Wm, Ws, g_w, Xv, Xs, g_x, M, N, K_lp, epilogue, out,
                                   stream)
        return out
    if out is None:
        out = _new(Xv, (M, N), out_dtype, stream)
    ss_sparse_gemm_nvfp4(Wv, Wm, Ws, g_w, Xv, Xs, g_x, M, N, K_lp, out, stream)
    return out


def dense_gemm_nvfp4(act, packed, M: int, N: int, out_dtype=torch.bfloat16, stream=None,
                     out=None, epilogue=None):
    Xv, Xs, g_x = act
    Wv, _, Ws, g_w = packed
    K_p = Xv.shape[1] * 2
    if epilogue is not None:
        out = epilogue._out(M, N, out_dtype, Xv, out, stream)
        ss_dense_gemm_nvfp4_fused(Xv, Xs, g_x, Wv, Ws, g_w, M, N, K_p, epilogue, out, stream)
        return out
    if out is None:
        out = _new(Xv, (M, N), out_dtype, stream)
    ss_dense_gemm_nvfp4(Xv, Xs, g_x, Wv, Ws, g_w, M, N, K_p, out, stream)
    return out


def linear_nvfp4(X: torch.Tensor, packed, pattern, out_dtype=torch.bfloat16, stream=None,
                 epilogue=None, out=None):
    """Y = X W^T in NVFP4: quantisation with one global scale for X + pair
    lift (blocks of 32 for a sparse weight, 16 for a dense one), then the
    block-scaled GEMM, with the fused epilogue if one is given.  out: the
    [M, N] output (a gated one [M, N/2])."""
    away = _away(X, stream)
    if away is not None:
        with away:
            return linear_nvfp4(X, packed, pattern, out_dtype, None, epilogue, out)
    p = _pattern(pattern)
    dense = p.group == 0
    (M, K), N = X.shape, packed[0].shape[0]
    _fits(M, N, K, _fp4_k_lp(p.keep, p.group, K), packed[0].shape[1] * (2 if dense else 4), out,
          epilogue)
    act = quant_lift_act_nvfp4(X, p, 16 if dense else 32, stream)
    if dense:
        return dense_gemm_nvfp4(act, packed, M, N, out_dtype, stream, out, epilogue)
    return sparse_gemm_nvfp4(packed, act, M, N, out_dtype, stream, out, epilogue)


# ------------------------------------------------------------------ fused epilogue
# The calls below check shapes, types and devices (ValueError) before the C
# call; they, linear and linear_nvfp4 run on the device of their tensors, on its
# current stream, whatever device is current.

def _call(where: str, index: int, *args) -> None:
    """The C function `where`, with device `index` current."""
    fn = getattr(lib(), where)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status != SS_OK:
        raise SSError(status, where)


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _index(t, name: str) -> int:
    """Index of the CUDA device that t is on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _arg(t, name: str, shape, dtypes, index: int):
    """Data pointer of a contiguous CUDA tensor on device `index` with that
    shape (None: any) and one of the types; None stays None."""
    if t is None:
        return None
    try:
        if t.get_device() == index and t.dtype in dtypes and (shape is None or t.shape == shape) \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if _index(t, name) != index:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} dtype {t.dtype} not supported")


def _need(t, name: str, shape, dtypes, index: int):
    if t is None:
        raise ValueError(f"{name} is required")
    return _arg(t, name, shape, dtypes, index)


@functools.lru_cache(maxsize=None)
def _pattern_of(keep: int, group: int) -> ss_pattern:
    return ss_pattern(keep, group)


@functools.lru_cache(maxsize=1024)
def _pattern_named(s: str) -> ss_pattern:
    return _pattern(s)


@functools.lru_cache(maxsize=4096)
def _k_lp(keep: int, group: int, K: int) -> int:
    return ss_slide_shape(_pattern_of(keep, group), K)[2]


@functools.lru_cache(maxsize=4096)
def _fp4_k_lp(keep: int, group: int, K: int) -> int:
    return ss_fp4_shape(_pattern_of(keep, group), K)[1]


def _fits(M, N, K, K_lp, weight_k_lp, out, epilogue) -> None:
    """An activation [M, K] (K_lp lifted) and an output, if one is given, against
    a weight of N rows of weight_k_lp: the products themselves take pointers."""
    if K_lp != weight_k_lp:
        raise ValueError(f"X has {K} columns, {K_lp} lifted; the weight has {weight_k_lp}")
    shape = (M, N // 2 if epilogue is not None and epilogue.gated else N)
    if out is not None and out.shape != shape:
        raise ValueError(f"out must have shape {shape}, got {tuple(out.shape)}")


def _pattern_k_lp(pattern, K: int):
    p = _pattern_named(pattern) if isinstance(pattern, str) else _pattern(pattern)
    return p, _k_lp(p.keep, p.group, K)


_FLOATS = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)
_BYTES = (torch.uint8,)
_IN = {torch.float32: SS_IN_F32, torch.bfloat16: SS_IN_BF16}


class Epilogue:
    """What a GEMM does to its output before the one rounding to Y's type, in
    fp32: v = dequantised product + bias; Y = act(v) + residual, or, gated,
    Y = act(gate) * up over weight rows in groups of 16 (eight gates, then
    the eight rows they multiply: see interleave_gate_up).

    bias [N], residual [M, N]: bf16 or fp32, whatever Y's type; act: "none",
    "relu", "silu", "gelu" (tanh form) or "gelu_erf".  The residual may be the
    output tensor itself.  A gated output is [M, N/2] and takes no residual."""

    __slots__ = ("bias", "act", "gated", "residual")

    def __init__(self, bias=None, act="none", gated=False, residual=None):
        if act not in ACTS:
            raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
        self.bias, self.act, self.gated, self.residual = bias, act, bool(gated), residual

    def _out(self, M, N, out_dtype, like, out, stream):
        if out is not None:
            return out
        return _new(like, (M, N // 2 if self.gated else N), out_dtype, stream)

    def _args(self, M, N, Y):
        """(ss_epilogue, Y's pointer, Y's device), checked against the product's shape."""
        d = _index(Y, "Y")
        y = _arg(Y, "Y", (M, N // 2 if self.gated else N), _FLOATS, d)
        b, r = self.bias, self.residual
        e = ss_epilogue(_arg(b, "bias", (N,), _FLOATS, d), _arg(r, "residual", (M, N), _FLOATS, d),
                        SS_IN_BF16 if b is None else _IN[b.dtype],
                        SS_IN_BF16 if r is None else _IN[r.dtype], ACTS[self.act], self.gated)
        return e, y, d


_STORED_8BIT = (torch.uint8, torch.int8, torch.float8_e4m3fn)
_STORED_BF16 = (torch.bfloat16,)


def _scale_arg(s, name, n, q, d):
    return None if q == SS_BF16 else _need(s, name, (n,), _F32, d)


def _bytes_arg(t, name, n, d):
    """Pointer of a byte tensor of any shape with n elements."""
    p = _need(t, name, None, _BYTES, d)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} bytes, got {t.numel()}")
    return p


def ss_sparse_gemm_fused(sparse_operand: int, Av, Am, s_a, B, s_b, M: int, N: int, K_lp: int, q,
                         epilogue: Epilogue, Y, stream=None) -> None:
    q = _qdtype(q)
    e, y, d = epilogue._args(M, N, Y)
    rows_a, rows_b = (M, N) if sparse_operand else (N, M)
    vals = _STORED_BF16 if q == SS_BF16 else _STORED_8BIT
    a = _need(Av, "Av", (rows_a, K_lp // 2), vals, d)
    m = _bytes_arg(Am, "Am", (rows_a + 127) // 128 * 16 * K_lp, d)
    b = _need(B, "B", (rows_b, K_lp), vals, d)
    sa, sb = _scale_arg(s_a, "s_a", rows_a, q, d), _scale_arg(s_b, "s_b", rows_b, q, d)
    _call("ss_sparse_gemm_fused", d, sparse_operand, a, m, sa, b, sb, M, N, K_lp, q,
          ctypes.byref(e), y, _out_dtype(Y), _raw_stream(stream, d))


def ss_dense_gemm_fused(Xq, s_x, Wq, s_w, M: int, N: int, K_p: int, q, epilogue: Epilogue, Y,
                        stream=None) -> None:
    q = _qdtype(q)
    e, y, d = epilogue._args(M, N, Y)
    vals = _STORED_BF16 if q == SS_BF16 else _STORED_8BIT
    x, w = _need(Xq, "Xq", (M, K_p), vals, d), _need(Wq, "Wq", (N, K_p), vals, d)
    sx, sw = _scale_arg(s_x, "s_x", M, q, d), _scale_arg(s_w, "s_w", N, q, d)
    _call("ss_dense_gemm_fused", d, x, sx, w, sw, M, N, K_p, q, ctypes.byref(e), y,
          _out_dtype(Y), _raw_stream(stream, d))


def _fp4_scales(s, name, rows, K_lp, block, d):
    return _bytes_arg(s, name, ss_fp4_scale_bytes(rows, K_lp, block), d)


def _global_scale(g, name, d):
    p = _need(g, name, None, _F32, d)
    if g.numel() < 1:
        raise ValueError(f"{name} is empty")
    return p


def ss_sparse_gemm_nvfp4_fused(Wv, Wm, Ws, g_w, Xv, Xs, g_x, M: int, N: int, K_lp: int,
                               epilogue: Epilogue, Y, stream=None) -> None:
    e, y, d = epilogue._args(M, N, Y)
    args = (_need(Wv, "Wv", (N, K_lp // 4), _BYTES, d),
            _bytes_arg(Wm, "Wm", ss_meta_bytes(N, K_lp // 2), d),
            _fp4_scales(Ws, "Ws", N, K_lp, 32, d), _global_scale(g_w, "g_w", d),
            _need(Xv, "Xv", (M, K_lp // 2), _BYTES, d), _fp4_scales(Xs, "Xs", M, K_lp, 32, d),
            _global_scale(g_x, "g_x", d))
    _call("ss_sparse_gemm_nvfp4_fused", d, *args, M, N, K_lp, ctypes.byref(e), y,
          _out_dtype(Y), _raw_stream(stream, d))


def ss_dense_gemm_nvfp4_fused(Xv, Xs, g_x, Wv, Ws, g_w, M: int, N: int, K_p: int,
                              epilogue: Epilogue, Y, stream=None) -> None:
    e, y, d = epilogue._args(M, N, Y)
    args = (_need(Xv, "Xv", (M, K_p // 2), _BYTES, d), _fp4_scales(Xs, "Xs", M, K_p, 16, d),
            _global_scale(g_x, "g_x", d), _need(Wv, "Wv", (N, K_p // 2), _BYTES, d),
            _fp4_scales(Ws, "Ws", N, K_p, 16, d), _global_scale(g_w, "g_w", d))
    _call("ss_dense_gemm_nvfp4_fused", d, *args, M, N, K_p, ctypes.byref(e), y,
          _out_dtype(Y), _raw_stream(stream, d))


def interleave_gate_up(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """The rows of two [F, ...] weights (or biases) as a gated product takes
    them: groups of eight gates, then their eight partners.  F must be a
    multiple of 8; compress the result as one weight of 2F rows."""
    if gate.shape != up.shape or gate.shape[0] % 8 != 0:
        raise ValueError("gate and up must have the same shape, with a multiple of 8 rows")
    F = gate.shape[0]
    both = torch.stack((gate.reshape(F // 8, 8, -1), up.reshape(F // 8, 8, -1)), dim=1)
    return both.reshape(2 * F, *gate.shape[1:])


# ------------------------------------------------------------------ around the products

def ss_norm_quant_lift_act(X, weight, eps: float, pattern, q, Xq_lift, s_x, stream=None) -> None:
    q = _qdtype(q)
    d = _index(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be a [M, K] CUDA tensor")
    M, K = X.shape
    p, K_lp = _pattern_k_lp(pattern, K)
    x = _arg(X, "X", None, _FLOATS, d)
    w = _need(weight, "weight", (K,), _FLOATS, d)
    xq = _need(Xq_lift, "Xq_lift", (M, K_lp), _STORED_BF16 if q == SS_BF16 else _STORED_8BIT, d)
    sx = _scale_arg(s_x, "s_x", M, q, d)
    _call("ss_norm_quant_lift_act", d, x, _IN[X.dtype], w, _IN[weight.dtype], eps, M, K, p, q,
          xq, sx, _raw_stream(stream, d))


def norm_quant_lift_act(X: torch.Tensor, weight: torch.Tensor, eps: float, pattern, q,
                        stream=None, out=None):
    """RMS norm of X's rows, quantised and lifted as quant_lift_act does;
    -> (Xq_lift [M, K_lp], s_x [M], or None for the bf16 tier)."""
    if out is None:
        M, K = X.shape
        s_x = None if _qdtype(q) == SS_BF16 else _new(X, (M,), torch.float32, stream)
        out = (_new(X, (M, _pattern_k_lp(pattern, K)[1]), _vals_dtype(q), stream), s_x)
    ss_norm_quant_lift_act(X, weight, eps, pattern, q, out[0], out[1], stream)
    return out


def ss_rope_frequencies(rot_dim: int, base: float, scaling: ss_rope_scaling | None = None):
    """-> (rot_dim / 2 frequencies as a list of floats, scale)."""
    if rot_dim < 2:
        raise SSError(SS_ERR_INVALID_ARG, "ss_rope_frequencies")
    f, s = (ctypes.c_double * (rot_dim // 2))(), ctypes.c_double()
    _check(lib().ss_rope_frequencies(int(rot_dim), float(base),
                                     None if scaling is None else ctypes.byref(scaling), f,
                                     ctypes.byref(s)), "ss_rope_frequencies")
    return list(f), s.value


def rope_frequencies(rot_dim: int, base: float = 10000.0, kind: str = "none", factor: float = 1.0,
                     original: float = 0.0, low: float = 1.0, high: float | None = None,
                     device="cuda"):
    """-> (frequencies [rot_dim/2] float64 on `device`, scale) for rope().
    kind: "none", "linear", "ntk", "llama3" or "yarn" (see ss_rope_scaling);
    high defaults to 4 turns for llama3 and 32 for yarn."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(ROPE_KINDS)}, got {kind!r}")
    if high is None:
        high = 4.0 if kind == "llama3" else 32.0
    s = ss_rope_scaling(ROPE_KINDS[kind], factor, original, low, high)
    f, scale = ss_rope_frequencies(rot_dim, base, s)
    return torch.tensor(f, dtype=torch.float64, device=device), scale


def _heads(x, y, name, T, D, dtype, d) -> ss_rope_heads:
    if not isinstance(x, torch.Tensor) or not isinstance(y, torch.Tensor):
        raise ValueError(f"{name} and its output must be CUDA tensors")
    sx, sy = x.shape, y.shape
    if not (x.get_device() == d == y.get_device() and x.dtype == dtype == y.dtype):
        raise ValueError(f"{name} and its output must be {dtype} on cuda:{d}, like q")
    if len(sx) != 3 or sx[0] != T or sx[2] != D or sx != sy:
        raise ValueError(f"{name} and its output must be [{T}, heads, {D}], got {tuple(sx)} "
                         f"and {tuple(sy)}")
    (st, sh, se), (ot, oh, oe) = x.stride(), y.stride()
    if se != 1 or oe != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    if (T > 1 and ot < 1) or (sx[1] > 1 and oh < 1):
        raise ValueError(f"{name}'s output: its elements overlap")
    return ss_rope_heads(x.data_ptr(), y.data_ptr(), sx[1], st, sh, ot, oh)


def ss_rope(q, k, positions, freqs, layout, scale: float, q_out, k_out, stream=None) -> None:
    d = _index(q, "q")
    if q.dim() != 3 or q.dtype not in _FLOATS:
        raise ValueError("q must be a [T, heads, head_dim] float32 or bfloat16 tensor")
    if (k is None) != (k_out is None):
        raise ValueError("k and its output go together")
    layout = ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    T, _, D = q.shape
    hq = _heads(q, q_out, "q", T, D, q.dtype, d)
    hk = None if k is None else ctypes.byref(_heads(k, k_out, "k", T, D, q.dtype, d))
    pos = _need(positions, "positions", (T,), _INTS, d)
    f = _need(freqs, "freqs", None, _F64, d)
    _call("ss_rope", d, ctypes.byref(hq), hk, _IN[q.dtype], pos, positions.dtype == torch.int64, f,
          scale, T, D, 2 * freqs.numel(), layout, _raw_stream(stream, d))


_INTS = (torch.int32, torch.int64)
_F64 = (torch.float64,)


def rope(q: torch.Tensor, k, positions: torch.Tensor, freqs: torch.Tensor, layout="half",
         scale: float = 1.0, stream=None, out=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (or None), which may be
    strided views into a projection's output; -> (q', k').  The first
    2 * len(freqs) elements of each head turn; freqs and scale come from
    rope_frequencies.  out = (q, k): in place."""
    if out is None:
        out = (_new(q, q.shape, q.dtype, stream),
               None if k is None else _new(k, k.shape, k.dtype, stream))
    ss_rope(q, k, positions, freqs, layout, scale, out[0], out[1], stream)
    return out


def project_qkv(X: torch.Tensor, packed, pattern, q, heads: int, kv_heads: int, positions, freqs,
                layout="half", scale: float = 1.0, norm=None, bias=None, stream=None):
    """The attention's inputs of a transformer layer: RMS norm of X (norm =
    (weight, eps) or None) fused into its quantisation, the fused query / key /
    value product with its bias, and rotary positions on the query and key
    heads in place.  The weight's rows are (heads + 2 kv_heads) heads of equal
    size.  -> q [M, heads, D], k, v [M, kv_heads, D], views of one tensor."""
    if stream is not None:
        with _as_current(stream, X):
            return project_qkv(X, packed, pattern, q, heads, kv_heads, positions, freqs, layout,
                               scale, norm, bias)
    N = packed[0].shape[0]
    if N % (heads + 2 * kv_heads) != 0:
        raise ValueError(f"{N} rows are not {heads} + 2 * {kv_heads} heads")
    Y = linear(X, packed, pattern, q, norm=norm,
               epilogue=None if bias is None else Epilogue(bias=bias))
    Y = Y.view(X.shape[0], heads + 2 * kv_heads, -1)
    yq, yk, yv = Y.split((heads, kv_heads, kv_heads), dim=1)
    rope(yq, yk, positions, freqs, layout, scale, out=(yq, yk))
    return yq, yk, yv


def feed_forward(X: torch.Tensor, packed_gate_up, packed_down, pattern, q, act="silu", norm=None,
                 stream=None):
    """The feed-forward half of a transformer layer, X + down(act(gate) * up)
    with gate, up of the RMS norm of X (norm = (weight, eps) or None):
    `packed_gate_up` = compress_weight(interleave_gate_up(W_gate, W_up)).  What
    the down projection takes is rounded to bf16 first, whatever X's type.
    -> [M, K] of X's type."""
    if stream is not None:
        with _as_current(stream, X):
            return feed_forward(X, packed_gate_up, packed_down, pattern, q, act, norm)
    h = linear(X, packed_gate_up, pattern, q, norm=norm, epilogue=Epilogue(act=act, gated=True))
    return linear(h, packed_down, pattern, q, X.dtype, epilogue=Epilogue(residual=X))
