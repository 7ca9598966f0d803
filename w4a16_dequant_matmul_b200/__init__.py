"""Python binding of libwq, the B200 (sm_100a) library for round-to-nearest group-wise INT4
weight quantization and the W4A16 dequant-matmul.

Argument marshalling only: every function forwards device pointers of torch tensors to the
C ABI declared in include/wq.h, on the current CUDA stream; all arithmetic runs in the
library's kernels. There is no CPU path: without libwq.so or a CUDA device the calls raise.

Functions carry the C names:
    wq_quantize_rtn_g128(W, w_bit=4, group=128, zero_point=True) -> (packed, S, Z)
    wq_quantize_rtn_per_tensor(W) -> (packed, S, Z)
    wq_pack_int4(codes) -> packed
    wq_dequant(packed, S, Z, group, out_dtype) -> W_hat
    wq_w4a16_gemm(X, packed, S, Z, group) -> Y
    wq_w8a16_gemm(X, codes, S) -> Y
    wq_channel_stat(A, stat) -> float32 [cols]      (WQ_STAT_ABSMAX / WQ_STAT_ABSMEAN)
    wq_smooth_scales(xmax, wmax, alpha) -> s
    wq_awq_scales(a_mag, alpha) -> s
    wq_quantize_rtn_scaled(W, s, group=128, zero_point=True) -> (packed, S, Z)
    wq_scale_activations(X, s) -> X / s
    wq_quantize_gptq(W, X, group=128, zero_point=True, damp=0.01) -> (packed, S, Z)
    wq_kv4_alloc(num_blocks, kv_heads, head_dim, group, block_size) -> cache
    wq_kv4_block_tables(ctx_lens, new_lens, free_blocks, tables, block_size, n_slots)
        -> (slots, q_starts, kv_lens, taken)
    wq_kv4_append(K, V, slots, cache, group)
    wq_kv4_read(cache, slots, head_dim, group, out_dtype) -> (K, V)
    wq_kv4_attention(Q, cache, tables, q_starts, kv_lens, max_q, group, ...) -> out
    wq_get_status() -> int
S and Z are returned as torch.float16 tensors (binary16 bit patterns in the C ABI).
A call given a `stream` runs there, and what it allocates (results, workspace) belongs to that
stream, as under torch.cuda.stream(stream).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

from ._build import LIB_PATH, build_library  # noqa: F401  (build_library re-exported)

__all__ = [
    "WQError", "lib", "status_name",
    "wq_version", "wq_status_string", "wq_quantize_rtn_g128", "wq_quantize_rtn_per_tensor",
    "wq_quantize_per_tensor_workspace_bytes", "wq_quantize_rtn_per_tensor_noalloc",
    "wq_pack_int4", "wq_dequant", "wq_w4a16_gemm",
    "wq_w8a16_gemm", "wq_get_status", "wq_selftest_bounded_wait",
    "wq_channel_stat", "wq_smooth_scales", "wq_awq_scales", "wq_quantize_rtn_scaled",
    "wq_scale_activations", "wq_quantize_gptq", "wq_gptq_workspace_bytes",
    "wq_kv4_alloc", "wq_kv4_cache_bytes", "wq_kv4_block_tables", "wq_kv4_append",
    "wq_kv4_read", "wq_kv4_attention", "wq_kv4_attention_workspace_bytes",
    "WQ_F32", "WQ_BF16", "WQ_F16", "WQ_U8", "WQ_I8", "WQ_STAT_ABSMAX", "WQ_STAT_ABSMEAN",
]

WQ_F32, WQ_BF16, WQ_F16, WQ_U8, WQ_I8 = 0, 1, 2, 3, 4
WQ_STAT_ABSMAX, WQ_STAT_ABSMEAN = 0, 1
STATUS_NAMES = {
    0: "WQ_OK", 1: "WQ_ERR_NULL", 2: "WQ_ERR_SHAPE", 3: "WQ_ERR_ALIGN", 4: "WQ_ERR_DTYPE",
    5: "WQ_ERR_UNSUPPORTED", 6: "WQ_ERR_CUDA", 7: "WQ_ERR_NONFINITE", 8: "WQ_ERR_TIMEOUT",
    9: "WQ_ERR_RANGE", 10: "WQ_ERR_NODEVICE", 11: "WQ_ERR_DEVICE",
}


class WQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_name(status)} ({_raw_status_string(status)})")


class _QParams(ctypes.Structure):
    _fields_ = [("w_bit", ctypes.c_int32), ("group", ctypes.c_int32),
                ("zero_point", ctypes.c_int32)]


# wq_kv4_cache and wq_kv4_attention_args, packed in one call each (the decode hot path)
_KV4_CACHE = struct.Struct("Pqiiii")
_KV4_ATTENTION = struct.Struct("PqqqPqiiiiPqqPPqPqqPPQiiiiif")

_LIB = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32

_SIGNATURES = {
    "wq_version": (_I32, []),
    "wq_status_string": (ctypes.c_char_p, [_I32]),
    "wq_quantize_rtn_g128": (_I32, [_P, _I32, _I64, _I64, _I64, ctypes.POINTER(_QParams), _P, _P,
                                    _P, _P]),
    "wq_quantize_per_tensor_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "wq_quantize_rtn_per_tensor": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P,
                                          ctypes.c_size_t, _P]),
    "wq_quantize_rtn_per_tensor_noalloc": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]),
    "wq_pack_int4": (_I32, [_P, _I64, _I64, _P, _P]),
    "wq_dequant": (_I32, [_P, _P, _P, _I64, _I64, _I32, _P, _I32, _P]),
    "wq_w4a16_gemm": (_I32, [_P, _I64, _I64, _P, _P, _P, _I64, _I64, _I32, _P, _I64, _P]),
    "wq_w8a16_gemm": (_I32, [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _I64, _P]),
    "wq_get_status": (_I32, [_P]),
    "wq_channel_stat": (_I32, [_P, _I32, _I64, _I64, _I64, _I32, _P, _P]),
    "wq_smooth_scales": (_I32, [_P, _P, _I64, ctypes.c_float, _P, _P]),
    "wq_awq_scales": (_I32, [_P, _I64, ctypes.c_float, _P, _P]),
    "wq_quantize_rtn_scaled": (_I32, [_P, _I32, _I64, _I64, _I64, _P, ctypes.POINTER(_QParams),
                                      _P, _P, _P, _P]),
    "wq_scale_activations": (_I32, [_P, _I64, _I64, _I64, _P, _P, _I64, _P]),
    "wq_gptq_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "wq_quantize_gptq": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _I64, _I64, ctypes.c_double,
                                ctypes.POINTER(_QParams), _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "wq_selftest_bounded_wait": (_I32, [ctypes.c_uint64, _I32, _P]),
    "wq_kv4_cache_bytes": (ctypes.c_size_t, [ctypes.c_char_p]),
    "wq_kv4_block_tables": (_I32, [_P, _P, _I64, _P, _I64, _I32, _P, _I64, _I64, _P, _I64, _P,
                                   _P, _P, _P]),
    "wq_kv4_append": (_I32, [_P, _P, _I32, _I64, _I64, _I64, _I64, _I64, _P, ctypes.c_char_p,
                             _P]),
    "wq_kv4_read": (_I32, [ctypes.c_char_p, _P, _I64, _P, _P, _I32, _P]),
    "wq_kv4_attention_workspace_bytes": (ctypes.c_size_t, []),
    "wq_kv4_attention": (_I32, [ctypes.c_char_p, _P]),
}


def lib() -> ctypes.CDLL:
    """The loaded libwq.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m w4a16_dequant_matmul_b200._build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def status_name(status: int) -> str:
    return STATUS_NAMES.get(int(status), f"status {status}")


def _raw_status_string(status: int) -> str:
    try:
        return lib().wq_status_string(int(status)).decode()
    except Exception:  # the library itself may be what failed to load
        return "?"


def _check(status: int, where: str) -> None:
    if status != 0:
        raise WQError(status, where)


def _stream(stream=None):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_RAW_STREAM = None


def _stream_handle(t, stream=None) -> int:
    """cudaStream_t (as an int) of `stream`, or of the current stream of t's device; the
    raw accessor avoids building a Stream object per call on the decode hot path."""
    global _RAW_STREAM
    if stream is not None:
        return stream.cuda_stream
    if _RAW_STREAM is None:
        import torch

        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    dev = t.get_device()
    if dev < 0:  # a host tensor: the library rejects it; any stream will do
        import torch

        dev = torch.cuda.current_device()
    return _RAW_STREAM(dev)


_GET_DEVICE = None


def _on_device(t):
    """A context that makes the CUDA device holding tensor t current for the call (the C
    library works on the current device and rejects other devices' memory); a no-op when
    it already is current, or when t is not a CUDA tensor."""
    global _GET_DEVICE
    d = t.get_device()
    if d < 0:
        return contextlib.nullcontext()
    import torch

    if _GET_DEVICE is None:
        _GET_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if _GET_DEVICE() == d:
        return contextlib.nullcontext()
    return torch.cuda.device(d)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _empty(shape, dtype, device, stream):
    """Memory for work on `stream` (None: the current one). It belongs to that stream, so that
    torch hands it, once let go, to later work of that stream only."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, name):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))


def _w_dtype(t):
    import torch

    if t.dtype == torch.float32:
        return WQ_F32
    if t.dtype == torch.bfloat16:
        return WQ_BF16
    raise TypeError("W must be float32 or bfloat16")


def wq_version() -> int:
    return int(lib().wq_version())


def wq_status_string(status: int) -> str:
    return _raw_status_string(status)


def wq_quantize_rtn_g128(W, w_bit: int = 4, group: int = 128, zero_point: bool = True,
                         packed=None, S=None, Z=None, stream=None):
    """Round-to-nearest quantization of W [N, K]. INT4 asymmetric ({4, g, True}) returns
    (packed uint8 [N, K/2], S fp16 [N, K/g], Z fp16 [N, K/g]); INT4 symmetric
    ({4, g, False}) the same, with codes q + 8 and every Z = 8; INT8 symmetric per channel
    ({8, K, False}) returns (codes int8 [N, K], S fp16 [N], None)."""
    import torch

    N, K = W.shape
    ldw = _rows(W, "W")
    dev = W.device
    if w_bit == 4:
        packed = _empty((N, K // 2), torch.uint8, dev, stream) if packed is None else packed
        G = K // group if group else 1
        S = _empty((N, G), torch.float16, dev, stream) if S is None else S
        Z = _empty((N, G), torch.float16, dev, stream) if Z is None else Z
    else:
        packed = _empty((N, K), torch.int8, dev, stream) if packed is None else packed
        S = _empty((N,), torch.float16, dev, stream) if S is None else S
    p = _QParams(w_bit, group, 1 if zero_point else 0)
    with _on_device(W):
        st = lib().wq_quantize_rtn_g128(_ptr(W), _w_dtype(W), N, K, ldw, ctypes.byref(p),
                                        _ptr(packed), _ptr(S), _ptr(Z), _stream(stream))
    _check(st, "wq_quantize_rtn_g128")
    return packed, S, Z


def wq_quantize_per_tensor_workspace_bytes(N: int, K: int) -> int:
    return int(lib().wq_quantize_per_tensor_workspace_bytes(N, K))


def wq_quantize_rtn_per_tensor(W, workspace=None, stream=None):
    """Per-tensor asymmetric INT4: returns (packed [N, K/2], S fp16 [1], Z fp16 [1])."""
    import torch

    N, K = W.shape
    ldw = _rows(W, "W")
    dev = W.device
    packed = _empty((N, K // 2), torch.uint8, dev, stream)
    S = _empty((1,), torch.float16, dev, stream)
    Z = _empty((1,), torch.float16, dev, stream)
    nbytes = wq_quantize_per_tensor_workspace_bytes(N, K)
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, dev, stream)
    with _on_device(W):
        st = lib().wq_quantize_rtn_per_tensor(_ptr(W), _w_dtype(W), N, K, ldw, _ptr(packed),
                                              _ptr(S), _ptr(Z), _ptr(workspace),
                                              workspace.numel() * workspace.element_size(),
                                              _stream(stream))
    _check(st, "wq_quantize_rtn_per_tensor")
    return packed, S, Z


def wq_quantize_rtn_per_tensor_noalloc(W, stream=None):
    """Per-tensor asymmetric INT4 without a workspace (for callers that cannot allocate
    device memory); the library's own fixed scratch array is used. Returns
    (packed [N, K/2], S fp16 [1], Z fp16 [1]). Output tensors are allocated here by torch
    only for convenience; C callers pass their own."""
    import torch

    N, K = W.shape
    ldw = _rows(W, "W")
    packed = _empty((N, K // 2), torch.uint8, W.device, stream)
    S = _empty((1,), torch.float16, W.device, stream)
    Z = _empty((1,), torch.float16, W.device, stream)
    with _on_device(W):
        st = lib().wq_quantize_rtn_per_tensor_noalloc(_ptr(W), _w_dtype(W), N, K, ldw,
                                                      _ptr(packed), _ptr(S), _ptr(Z),
                                                      _stream(stream))
    _check(st, "wq_quantize_rtn_per_tensor_noalloc")
    return packed, S, Z


def wq_pack_int4(codes, packed=None, stream=None):
    """codes uint8 [N, K] in [0, 15] -> packed uint8 [N, K/2]."""
    import torch

    N, K = codes.shape
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    packed = _empty((N, K // 2), torch.uint8, codes.device, stream) if packed is None else packed
    with _on_device(codes):
        st = lib().wq_pack_int4(_ptr(codes), N, K, _ptr(packed), _stream(stream))
    _check(st, "wq_pack_int4")
    return packed


def wq_dequant(packed, S, Z, group: int = 128, out_dtype=None, out=None, stream=None):
    """W_hat = S'(q - Z) as float32 (exact) or bfloat16 [N, K]."""
    import torch

    out_dtype = torch.float32 if out_dtype is None else out_dtype
    N, K2 = packed.shape
    K = 2 * K2
    code = WQ_F32 if out_dtype == torch.float32 else WQ_BF16 if out_dtype == torch.bfloat16 else -1
    out = _empty((N, K), out_dtype, packed.device, stream) if out is None else out
    with _on_device(packed):
        st = lib().wq_dequant(_ptr(packed), _ptr(S), _ptr(Z), N, K, group, _ptr(out), code,
                              _stream(stream))
    _check(st, "wq_dequant")
    return out


_GEMM = None


def wq_w4a16_gemm(X, packed, S, Z, group: int = 128, Y=None, stream=None):
    """Y [M, N] bf16 = X [M, K] bf16 @ W_hat^T, fp32 accumulation. (The decode hot path:
    raw integer pointers and a cached function handle keep the per-call host cost low.)"""
    global _GEMM
    if _GEMM is None:
        _GEMM = lib().wq_w4a16_gemm
    M, K = X.shape
    N = packed.shape[0]
    ldx = _rows(X, "X")
    if Y is None:
        import torch

        Y = _empty((M, N), torch.bfloat16, X.device, stream)
    ldy = _rows(Y, "Y")
    with _on_device(X):
        st = _GEMM(X.data_ptr(), M, ldx, packed.data_ptr(), S.data_ptr(), Z.data_ptr(), N, K,
                   group, Y.data_ptr(), ldy, _stream_handle(X, stream))
    if st != 0:
        raise WQError(st, "wq_w4a16_gemm")
    return Y


def wq_w8a16_gemm(X, codes, S, Y=None, stream=None):
    """Y [M, N] bf16 = X [M, K] bf16 @ (s' q)^T with INT8 per-channel weights."""
    import torch

    M, K = X.shape
    N = codes.shape[0]
    ldx = _rows(X, "X")
    Y = _empty((M, N), torch.bfloat16, X.device, stream) if Y is None else Y
    ldy = _rows(Y, "Y")
    with _on_device(X):
        st = lib().wq_w8a16_gemm(_ptr(X), M, ldx, _ptr(codes), _ptr(S), N, K, _ptr(Y), ldy,
                                 _stream(stream))
    _check(st, "wq_w8a16_gemm")
    return Y


def wq_channel_stat(A, stat: int = WQ_STAT_ABSMAX, out=None, stream=None):
    """Per-column max |A_ij| (WQ_STAT_ABSMAX) or mean |A_ij| (WQ_STAT_ABSMEAN) of A [rows,
    cols] (float32 or bfloat16) -> float32 [cols]."""
    import torch

    rows, cols = A.shape
    lda = _rows(A, "A")
    out = _empty((cols,), torch.float32, A.device, stream) if out is None else out
    with _on_device(A):
        st = lib().wq_channel_stat(_ptr(A), _w_dtype(A), rows, cols, lda, int(stat), _ptr(out),
                                   _stream(stream))
    _check(st, "wq_channel_stat")
    return out


def wq_smooth_scales(xmax, wmax, alpha: float = 0.5, out=None, stream=None):
    """SmoothQuant factors s_j = xmax_j^alpha / wmax_j^(1 - alpha), float32 [K]."""
    import torch

    K = xmax.shape[0]
    out = _empty((K,), torch.float32, xmax.device, stream) if out is None else out
    with _on_device(xmax):
        st = lib().wq_smooth_scales(_ptr(xmax), _ptr(wmax), K, float(alpha), _ptr(out),
                                    _stream(stream))
    _check(st, "wq_smooth_scales")
    return out


def wq_awq_scales(a_mag, alpha: float, out=None, stream=None):
    """AWQ factors a_j^alpha / sqrt(max * min), float32 [K]."""
    import torch

    K = a_mag.shape[0]
    out = _empty((K,), torch.float32, a_mag.device, stream) if out is None else out
    with _on_device(a_mag):
        st = lib().wq_awq_scales(_ptr(a_mag), K, float(alpha), _ptr(out), _stream(stream))
    _check(st, "wq_awq_scales")
    return out


def wq_quantize_rtn_scaled(W, s, group: int = 128, zero_point: bool = True, packed=None,
                           S=None, Z=None, stream=None):
    """RTN INT4 of W diag(s) (W [N, K] float32 or bfloat16, s float32 [K]): returns
    (packed uint8 [N, K/2], S fp16 [N, K/g], Z fp16 [N, K/g]) as wq_quantize_rtn_g128."""
    import torch

    N, K = W.shape
    ldw = _rows(W, "W")
    dev = W.device
    G = K // group if group else 1
    packed = _empty((N, K // 2), torch.uint8, dev, stream) if packed is None else packed
    S = _empty((N, G), torch.float16, dev, stream) if S is None else S
    Z = _empty((N, G), torch.float16, dev, stream) if Z is None else Z
    p = _QParams(4, group, 1 if zero_point else 0)
    with _on_device(W):
        st = lib().wq_quantize_rtn_scaled(_ptr(W), _w_dtype(W), N, K, ldw, _ptr(s),
                                          ctypes.byref(p), _ptr(packed), _ptr(S), _ptr(Z),
                                          _stream(stream))
    _check(st, "wq_quantize_rtn_scaled")
    return packed, S, Z


def wq_scale_activations(X, s, out=None, stream=None):
    """X / s per column (X [M, K] bfloat16, s float32 [K]) -> bfloat16 [M, K]; out may be
    X itself."""
    import torch

    M, K = X.shape
    ldx = _rows(X, "X")
    out = _empty((M, K), torch.bfloat16, X.device, stream) if out is None else out
    ldo = _rows(out, "out")
    with _on_device(X):
        st = lib().wq_scale_activations(_ptr(X), M, K, ldx, _ptr(s), _ptr(out), ldo,
                                        _stream(stream))
    _check(st, "wq_scale_activations")
    return out


def wq_gptq_workspace_bytes(N: int, K: int) -> int:
    return int(lib().wq_gptq_workspace_bytes(N, K))


def wq_quantize_gptq(W, X, group: int = 128, zero_point: bool = True, damp: float = 0.01,
                     workspace=None, stream=None):
    """GPTQ of W [N, K] (float32 or bfloat16) on calibration activations X [T, K] (bfloat16):
    returns (packed uint8 [N, K/2], S fp16 [N, K/g], Z fp16 [N, K/g]) in the RTN format."""
    import torch

    N, K = W.shape
    T = X.shape[0]
    ldw = _rows(W, "W")
    ldx = _rows(X, "X")
    dev = W.device
    packed = _empty((N, K // 2), torch.uint8, dev, stream)
    S = _empty((N, K // group), torch.float16, dev, stream)
    Z = _empty((N, K // group), torch.float16, dev, stream)
    nbytes = wq_gptq_workspace_bytes(N, K)
    if workspace is None:
        workspace = _empty((max(nbytes, 16),), torch.uint8, dev, stream)
    p = _QParams(4, group, 1 if zero_point else 0)
    with _on_device(W):
        st = lib().wq_quantize_gptq(_ptr(W), _w_dtype(W), N, K, ldw, _ptr(X), T, ldx,
                                    float(damp), ctypes.byref(p), _ptr(packed), _ptr(S), _ptr(Z),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check(st, "wq_quantize_gptq")
    return packed, S, Z


# The 4-bit KV cache calls are made once or more a decode step on tensors of a few KB, so what
# the host spends on them counts: names of torch and the library's functions are looked up
# once, and arguments travel packed.
_KV4 = None


class _Kv4Names:
    """torch's names and the library's functions that the calls below use."""

    def __init__(self):
        import torch

        self.int32, self.uint8, self.float32 = torch.int32, torch.uint8, torch.float32
        self.empty = torch.empty_strided
        self.code = {torch.bfloat16: WQ_BF16, torch.float16: WQ_F16}
        self.out_code = {torch.float32: WQ_F32, torch.bfloat16: WQ_BF16, torch.float16: WQ_F16}
        self.device, self.on_stream = torch.cuda.device, torch.cuda.stream
        self.current_device = getattr(torch._C, "_cuda_getDevice", None) or \
            torch.cuda.current_device
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        self.workspace_bytes = {}  # by device
        handle = lib()
        self.block_tables = handle.wq_kv4_block_tables
        self.append = handle.wq_kv4_append
        self.read = handle.wq_kv4_read
        self.attention = handle.wq_kv4_attention


def _kv4():
    global _KV4
    if _KV4 is None:
        _KV4 = _Kv4Names()
    return _KV4


def _kv4_stream(k, t, stream):
    """Handle of the current stream where `stream` (None: any) and t's device are the current
    ones; else a context that makes them so, in which the caller calls itself again without a
    stream. What a call allocates (results, workspace) so belongs to the stream that it runs on:
    torch hands memory that is let go only to later work of the stream that it belongs to."""
    d = t.get_device()
    if d < 0:  # a host tensor: the library rejects it; any stream will do
        return 0
    if stream is not None:
        if stream.device.index != d:
            raise ValueError(f"the stream is of {stream.device}, the tensors of device {d}")
        if d != k.current_device() or stream.cuda_stream != k.raw_stream(d):
            return k.on_stream(stream)
    elif d != k.current_device():
        return k.device(t.device)
    return k.raw_stream(d)


def _kv4_bad_ints(t, name, n):
    if t.dtype is not _kv4().int32:
        raise TypeError(f"{name} must be int32")
    raise ValueError(f"{name} must be contiguous, of shape {n}, not {tuple(t.shape)}")


def _kv4_heads(t, name):
    """(tokens, heads, head_dim, token stride, head stride) of a [T, heads, head_dim] tensor."""
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return n, h, d, st if n > 1 else 0, sh if h > 1 else 0


def _kv4_code(t, name):
    code = _kv4().code.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float16")
    return code


def _kv4_tables(t, B):
    """Width and row stride of block tables int32 [B, width]."""
    if t.dtype is not _kv4().int32 or t.dim() != 2 or t.shape[0] != B:
        raise ValueError("tables must be int32 [B, width]")
    if t.is_contiguous():
        width = t.shape[1]
        return width, width
    return t.shape[1], _rows(t, "tables")


def _kv4_cache(cache, head_dim, group):
    """The fields of wq_kv4_cache for a cache tensor of wq_kv4_alloc."""
    group = head_dim if group is None else group
    if cache.dtype is not _kv4().uint8 or cache.dim() != 3 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 [num_blocks, kv_heads, bytes] tensor")
    n, h, chunk = cache.shape
    row = head_dim + 8 * (head_dim // group) if group > 0 else 0
    if row <= 0 or chunk % row:
        raise ValueError(f"a cache with {chunk} bytes a chunk is not one of head_dim {head_dim}, "
                         f"group {group}")
    return cache.data_ptr(), n, h, head_dim, group, chunk // row


def wq_kv4_cache_bytes(num_blocks: int, kv_heads: int, head_dim: int, group: int = None,
                       block_size: int = 64) -> int:
    """Bytes of a 4-bit KV cache; 0 if the description is not supported."""
    group = head_dim if group is None else group
    return int(lib().wq_kv4_cache_bytes(
        _KV4_CACHE.pack(0, num_blocks, kv_heads, head_dim, group, block_size)))


def wq_kv4_alloc(num_blocks: int, kv_heads: int, head_dim: int, group: int = None,
                 block_size: int = 64, device="cuda"):
    """Memory of a 4-bit KV cache: uint8 [num_blocks, kv_heads, bytes of a block of a head], not
    initialised. group defaults to head_dim (one scale a row)."""
    import torch

    one = wq_kv4_cache_bytes(1, kv_heads, head_dim, group, block_size)
    if one == 0 or (num_blocks > 0 and wq_kv4_cache_bytes(num_blocks, kv_heads, head_dim, group,
                                                          block_size) == 0):
        raise WQError(5, "wq_kv4_alloc")
    return torch.empty((num_blocks, kv_heads, one // kv_heads), dtype=torch.uint8, device=device)


def wq_kv4_block_tables(ctx_lens, new_lens, free_blocks, tables, block_size: int, n_slots: int,
                        stream=None):
    """Block tables and slot map of one step: enters the blocks that the requests' new tokens
    need, taken from free_blocks in order, into `tables` (int32 [B, width], in place) and
    returns (slots int32 [n_slots], q_starts int32 [B + 1], kv_lens int32 [B], taken int32 [1]).
    ctx_lens, new_lens: int32 [B], tokens held and tokens to come. Slots behind the last new
    token are -1."""
    k = _KV4 or _kv4()
    handle = _kv4_stream(k, ctx_lens, stream)
    if handle.__class__ is not int:
        with handle:
            return wq_kv4_block_tables(ctx_lens, new_lens, free_blocks, tables, block_size,
                                       n_slots)
    i32 = k.int32
    B = ctx_lens.shape[0]
    if ctx_lens.dtype is not i32 or ctx_lens.dim() != 1 or not ctx_lens.is_contiguous():
        _kv4_bad_ints(ctx_lens, "ctx_lens", (B,))
    if new_lens.dtype is not i32 or new_lens.shape != (B,) or not new_lens.is_contiguous():
        _kv4_bad_ints(new_lens, "new_lens", (B,))
    if free_blocks.dtype is not i32 or free_blocks.dim() != 1 or not free_blocks.is_contiguous():
        _kv4_bad_ints(free_blocks, "free_blocks", ("n",))
    width, ld = _kv4_tables(tables, B)
    out = k.empty((n_slots + 2 * B + 2,), (1,), dtype=i32, device=ctx_lens.device)
    slots, q_starts, kv_lens, taken = out.split_with_sizes((n_slots, B + 1, B, 1))
    at = out.data_ptr()
    st = k.block_tables(ctx_lens.data_ptr(), new_lens.data_ptr(), B, free_blocks.data_ptr(),
                        free_blocks.shape[0], block_size, tables.data_ptr(), width, ld, at,
                        n_slots, at + 4 * n_slots, at + 4 * (n_slots + B + 1),
                        at + 4 * (n_slots + 2 * B + 1), handle)
    if st != 0:
        raise WQError(st, "wq_kv4_block_tables")
    return slots, q_starts, kv_lens, taken


def wq_kv4_append(K, V, slots, cache, group: int = None, stream=None) -> None:
    """Quantize keys and values [T, kv_heads, head_dim] (bfloat16 or float16, any token and head
    strides) into slots (int32 [T], negative: skipped) of the cache."""
    k = _KV4 or _kv4()
    handle = _kv4_stream(k, K, stream)
    if handle.__class__ is not int:
        with handle:
            return wq_kv4_append(K, V, slots, cache, group)
    T, h, d, kt, kh = _kv4_heads(K, "K")
    if V.shape != K.shape or V.dtype is not K.dtype:
        raise ValueError("K and V must have one shape and dtype")
    _, _, _, vt, vh = _kv4_heads(V, "V")
    if slots.dtype is not k.int32 or slots.shape != (T,) or not slots.is_contiguous():
        _kv4_bad_ints(slots, "slots", (T,))
    c = _kv4_cache(cache, d, group)
    if c[2] != h:
        raise ValueError(f"the cache has {c[2]} KV heads, K has {h}")
    st = k.append(K.data_ptr(), V.data_ptr(), _kv4_code(K, "K"), T, kt, kh, vt, vh,
                  slots.data_ptr(), _KV4_CACHE.pack(*c), handle)
    if st != 0:
        raise WQError(st, "wq_kv4_append")


def wq_kv4_read(cache, slots, head_dim: int, group: int = None, out_dtype=None, stream=None):
    """Values S'(q - Z) stored in slots (int32 [T]; zeros for negative ones): (K, V), each
    [T, kv_heads, head_dim] float32 (exact), bfloat16 or float16."""
    k = _KV4 or _kv4()
    handle = _kv4_stream(k, cache, stream)
    if handle.__class__ is not int:
        with handle:
            return wq_kv4_read(cache, slots, head_dim, group, out_dtype)
    out_dtype = k.float32 if out_dtype is None else out_dtype
    if slots.dtype is not k.int32 or slots.dim() != 1 or not slots.is_contiguous():
        _kv4_bad_ints(slots, "slots", ("T",))
    c = _kv4_cache(cache, head_dim, group)
    T, h = slots.shape[0], c[2]
    shape, strides, dev = (T, h, head_dim), (h * head_dim, head_dim, 1), cache.device
    K = k.empty(shape, strides, dtype=out_dtype, device=dev)
    V = k.empty(shape, strides, dtype=out_dtype, device=dev)
    st = k.read(_KV4_CACHE.pack(*c), slots.data_ptr(), T, K.data_ptr(), V.data_ptr(),
                k.out_code.get(out_dtype, -1), handle)
    if st != 0:
        raise WQError(st, "wq_kv4_read")
    return K, V


def wq_kv4_attention_workspace_bytes() -> int:
    return int(lib().wq_kv4_attention_workspace_bytes())


def wq_kv4_attention(Q, cache, tables, q_starts, kv_lens, max_q: int, group: int = None,
                     scale: float = None, causal: bool = True, window: int = 0, out=None,
                     return_lse: bool = False, workspace=None, stream=None):
    """Attention of Q [T, heads, head_dim] (bfloat16 or float16) over the cache: rows
    q_starts[b] .. q_starts[b + 1] - 1 are the last tokens of request b, whose kv_lens[b] tokens
    lie in the blocks of tables[b]. Returns out (Q's shape and type), or (out, lse float32
    [T, heads]). scale defaults to head_dim ** -0.5; max_q: the largest number of rows of a
    request; window > 0: each row sees the last `window` keys only (table entries of blocks that
    no row sees are not read). Rows outside q_starts are left as they were."""
    k = _KV4 or _kv4()
    handle = _kv4_stream(k, Q, stream)
    if handle.__class__ is not int:
        with handle:
            return wq_kv4_attention(Q, cache, tables, q_starts, kv_lens, max_q, group, scale,
                                    causal, window, out, return_lse, workspace)
    T, heads, d, qt, qh = _kv4_heads(Q, "Q")
    c = _kv4_cache(cache, d, group)
    B = kv_lens.shape[0]
    if kv_lens.dtype is not k.int32 or kv_lens.dim() != 1 or not kv_lens.is_contiguous():
        _kv4_bad_ints(kv_lens, "kv_lens", (B,))
    if q_starts.dtype is not k.int32 or q_starts.shape != (B + 1,) or not q_starts.is_contiguous():
        _kv4_bad_ints(q_starts, "q_starts", (B + 1,))
    width, ld = _kv4_tables(tables, B)
    dev = Q.device
    if out is None:
        ot, oh = heads * d, d
        out = k.empty((T, heads, d), (ot, oh, 1), dtype=Q.dtype, device=dev)
    else:
        if out.shape != Q.shape or out.dtype is not Q.dtype:
            raise ValueError("out must have Q's shape and dtype")
        _, _, _, ot, oh = _kv4_heads(out, "out")
    lse = None
    if return_lse:
        lse = k.empty((T, heads), (heads, 1), dtype=k.float32, device=dev)
    if workspace is None:
        n = k.workspace_bytes.get(dev)
        if n is None:
            n = k.workspace_bytes[dev] = wq_kv4_attention_workspace_bytes()
        workspace = k.empty((n,), (1,), dtype=k.uint8, device=dev)
    else:
        n = workspace.numel() * workspace.element_size()
    args = _KV4_ATTENTION.pack(
        Q.data_ptr(), T, qt, qh, *c, tables.data_ptr(), width, ld, q_starts.data_ptr(),
        kv_lens.data_ptr(), B, out.data_ptr(), ot, oh, 0 if lse is None else lse.data_ptr(),
        workspace.data_ptr(), n, _kv4_code(Q, "Q"), heads, int(max_q), 1 if causal else 0,
        int(window), d ** -0.5 if scale is None else float(scale))
    st = k.attention(args, handle)
    if st != 0:
        raise WQError(st, "wq_kv4_attention")
    return (out, lse) if return_lse else out


def wq_selftest_bounded_wait(limit_ns: int = 20_000_000, spin: bool = True, stream=None) -> None:
    """Launch the failure-detection self-test (a bounded wait that runs out); the next
    wq_get_status() then returns WQ_ERR_TIMEOUT (8)."""
    _check(lib().wq_selftest_bounded_wait(int(limit_ns), 1 if spin else 0, _stream(stream)),
           "wq_selftest_bounded_wait")


def wq_get_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(lib().wq_get_status(_stream(stream)))
