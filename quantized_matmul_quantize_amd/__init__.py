"""Group-wise INT4 weight quantization and quantized matmuls for AMD MI355X (gfx950).

Thin Python binding over the C ABI of ``libqmm.so`` (declared in
``include/qmm.h``).  It only marshals arguments: it checks every tensor's
shape, dtype, device and layout against the call (``ValueError`` before any
launch), allocates output tensors with torch (device memory), passes raw
device pointers and the current HIP stream, and turns a non-zero status into
``QmmError``.  Every computation runs in the library's hand-written HIP
kernels; there is no fallback path, and the functions raise if the library
has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import Optional, Sequence, Tuple

import torch

from .kv_pages import KvPages

__all__ = [
    "QmmError", "lib", "library_path", "F32", "F16", "BF16", "I32", "GROUP", "SQ_STATIC_SCRATCH_BYTES",
    "w4_sizes", "wq_sizes", "quantize_groupwise", "quantize_groupwise_symmetric", "quantize_groupwise_ex",
    "dequantize", "dequantize_ex", "w4a16_gemv", "w4a16_gemm", "wxa16_gemv", "wxa16_gemm",
    "w4_repack_from_plain", "w4_repack_to_plain", "w8a16_gemv",
    "sq_smooth_factors", "sq_quantize_weight", "sq_quantize_activation", "sq_quantize_activation_per_tensor",
    "sq_int8_gemm", "sq_workspace_bytes", "smooth_quant_w8a8_gemm", "smooth_quant_w8a8_gemm_noalloc",
    "fp8_quantize", "fp8_gemm", "fp8_w8a8_gemm",
    "llm_int8_outliers", "llm_int8_workspace_bytes", "llm_int8_gemm", "awq_workspace_bytes", "awq_search", "stream_read",
    "kv4_cache", "kv4_page_bytes", "kv4_append", "kv4_read", "kv4_copy_pages", "kv4_attention_workspace_bytes",
    "kv4_attention", "rope_frequencies", "rope_table", "qk_norm_rope", "KvPages",
]

F32, F16, BF16, I32 = 0, 1, 2, 3
GROUP = 128
_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16, torch.int32: I32}
_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_HALVES = (torch.bfloat16, torch.float16)

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libqmm.so")

# Device scratch of smooth_quant_w8a8_gemm_noalloc (QMM_SQ_STATIC_SCRATCH_BYTES).
SQ_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024 + 64 * 1024


class QmmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().qmm_status_string(status).decode() if status else "ok"
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


_lib: Optional[ctypes.CDLL] = None

# name -> argument types of the C ABI
_P, _I64, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "qmm_status_string": ([_I], ctypes.c_char_p),
    "qmm_version": ([], _I),
    "qmm_w4_sizes": ([_I64, _I64, _I, _P, _P, _P], _I),
    "qmm_wq_sizes": ([_I64, _I64, _I, _I, _I, _P, _P, _P], _I),
    "quantize_groupwise": ([_P, _I, _I64, _I64, _I, _I, _P, _P, _P, _P], _I),
    "quantize_groupwise_symmetric": ([_P, _I, _I64, _I64, _I, _I, _P, _P, _P, _P], _I),
    "quantize_groupwise_ex": ([_P, _I, _I64, _I64, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "dequantize": ([_P, _P, _P, _I64, _I64, _I, _I, _P, _I, _P], _I),
    "dequantize_ex": ([_P, _P, _P, _I64, _I64, _I, _I, _I, _P, _I, _P], _I),
    "w4a16_gemv": ([_P, _P, _P, _I64, _I64, _I, _P, _I, _I64, _P, _I, _P], _I),
    "w4a16_gemm": ([_P, _P, _P, _I64, _I64, _I, _P, _I, _I64, _P, _I, _P], _I),
    "wxa16_gemv": ([_P, _P, _P, _I64, _I64, _I, _I, _I, _P, _I, _I64, _P, _I, _P], _I),
    "wxa16_gemm": ([_P, _P, _P, _I64, _I64, _I, _I, _I, _P, _I, _I64, _P, _I, _P], _I),
    "qmm_w4_repack_from_plain": ([_P, _P, _I64, _I64, _P], _I),
    "qmm_w4_repack_to_plain": ([_P, _P, _I64, _I64, _P], _I),
    "w8a16_gemv": ([_P, _P, _I64, _I64, _P, _I, _I64, _P, _I, _P], _I),
    "sq_smooth_factors": ([_P, _I, _I64, _P, _I, _I64, _I64, _F, _P, _P, _P, _P], _I),
    "sq_quantize_weight": ([_P, _I, _P, _I64, _I64, _P, _P, _P], _I),
    "sq_quantize_activation": ([_P, _I, _P, _I64, _I64, _P, _P, _P], _I),
    "sq_quantize_activation_per_tensor": ([_P, _I, _P, _I64, _I64, _P, _P, _P], _I),
    "sq_int8_gemm": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "sq_workspace_bytes": ([_I64, _I64], _SZ),
    "smooth_quant_w8a8_gemm": ([_P, _I, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P, _SZ, _P], _I),
    "smooth_quant_w8a8_gemm_noalloc": ([_P, _I, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "fp8_quantize": ([_P, _I, _I64, _I64, _I, _P, _P, _P], _I),
    "fp8_gemm": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "fp8_w8a8_gemm": ([_P, _I, _P, _P, _I64, _I64, _I64, _P, _I, _P, _SZ, _P], _I),
    "llm_int8_outliers": ([_P, _I, _I64, _I64, _F, _I64, _P, _P, _P, _P], _I),
    "llm_int8_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "awq_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "qmm_stream_read": ([_P, _SZ, _P, _P], _I),
    "awq_search": ([_P, _I, _P, _I, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "llm_int8_gemm": ([_P, _I, _P, _P, _I64, _I64, _I64, _F, _I64, _P, _I, _P, _P, _SZ, _P], _I),
    "kv4_page_bytes": ([_I64, _I64, _I64, _I], _SZ),
    "kv4_append": ([_P, _I64, _I64, _P, _I64, _I64, _I, _I64, _P, _P, _I64, _I64, _I64, _I64, _I, _P], _I),
    "kv4_read": ([_P, _I64, _I64, _I64, _I64, _I, _P, _I64, _P, _P, _I, _P], _I),
    "kv4_copy_pages": ([_P, _I64, _I64, _I64, _P, _P, _I64, _P], _I),
    "kv4_attention_workspace_bytes": ([_I64] * 6 + [_I] + [_I64] * 3, _SZ),
    "kv4_attention": ([_P, _I64, _I64, _I, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64,
                       _I, _F, _I64, _I64, _P, _P, _P, _SZ, _P], _I),
    "qk_norm_rope": ([_P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I, _I64, _I64, _P, _P, _I64, _I64, _I, _P, _P, _I,
                      _F, _P, _P, _P], _I),
    "rope_table": ([_P, _I64, _I64, ctypes.c_double, _P, _P], _I),
}
# The calls of a decode step with their arguments as one block of 8-byte words (include/qmm_blocks.h): ctypes converts
# one argument and not up to 27 (kv4_attention: 3.8 us a call by arguments, 0.7 by a block).
_BLOCKS = {name: struct.Struct("=" + "".join("d" if t is _F else "q" for t in _SIGS[name][0]))
           for name in ("kv4_append", "kv4_read", "kv4_copy_pages", "kv4_attention", "qk_norm_rope")}
_SIGS.update({name + "_block": ([ctypes.c_char_p], _I) for name in _BLOCKS})


def lib() -> ctypes.CDLL:
    """The loaded libqmm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise ImportError(f"{library_path} is missing: build it with __graft_entry__.build() "
                              "(python -m quantized_matmul_quantize_amd._build)")
        l = ctypes.CDLL(library_path)
        for name, (argtypes, restype) in _SIGS.items():
            fn = getattr(l, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = l
    return _lib


def _call(name: str, *args) -> None:
    st = getattr(lib(), name)(*args)
    if st != 0:
        raise QmmError(name, st)


def _call_block(name: str, *args) -> None:
    st = getattr(lib(), name + "_block")(_BLOCKS[name].pack(*args))
    if st != 0:
        raise QmmError(name, st)


def _ptr0(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor):
    return torch._C._cuda_getCurrentRawStream(t.get_device())     # without a Stream object around it


def _dt(dtype: torch.dtype) -> int:
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    return _DT[dtype]


def _req(t, name: str, dtypes: Sequence[torch.dtype], shape: Optional[Tuple] = None,
         ndim: Optional[int] = None) -> None:
    """Check one operand's dtype and shape (None entries are free) or number
    of dimensions.  Raises ValueError."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {list(dtypes)}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, has shape {tuple(t.shape)}")
    if shape is not None:
        if t.dim() != len(shape) or any(s is not None and int(a) != int(s) for a, s in zip(t.shape, shape)):
            raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")


def _place(**tensors) -> torch.device:
    """After every shape and dtype check: all operands on one GPU, contiguous.
    Returns their device.  None entries (optional operands) are skipped."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return dev


def _out(out: Optional[torch.Tensor], shape: Tuple, dtype: torch.dtype, name: str = "out") -> None:
    if out is not None:
        _req(out, name, (dtype,), shape=shape)


def _alloc(out: Optional[torch.Tensor], shape: Tuple, dtype: torch.dtype, device) -> torch.Tensor:
    return out if out is not None else torch.empty(shape, dtype=dtype, device=device)


def _sdt(scale_dtype: torch.dtype) -> int:
    if scale_dtype not in (torch.float32, torch.float16):
        raise ValueError(f"scale_dtype must be torch.float32 or torch.float16, not {scale_dtype}")
    return _DT[scale_dtype]


def _groups(K: int, group: int) -> int:
    if group <= 0 or K % group:
        raise ValueError(f"K = {K} is not a multiple of the group size {group}")
    return K // group


def _code_cols(K: int, bits: int) -> int:
    return K * bits // 8


def _zero_cols(G: int, bits: int) -> int:
    return (G + 1) // 2 if bits <= 4 else G


def _k_from_codes(codes: torch.Tensor, bits: int) -> int:
    if bits not in (3, 4, 8):
        raise ValueError(f"bits must be 3, 4 or 8, not {bits}")
    if codes.dim() != 2 or (codes.shape[1] * 8) % bits:
        raise ValueError(f"codes of shape {tuple(codes.shape)} do not hold {bits}-bit codes")
    return codes.shape[1] * 8 // bits


def _check_format(codes, scales, zeros, group: int, bits: int, scale_dtype: torch.dtype):
    """Shapes and dtypes of the stored-format operands of one weight matrix; returns (N, K)."""
    if not isinstance(codes, torch.Tensor):
        raise ValueError("codes must be a torch.Tensor")
    K = _k_from_codes(codes, bits)
    N = codes.shape[0]
    G = _groups(K, group)
    _req(codes, "codes", (torch.uint8,), shape=(N, _code_cols(K, bits)))
    _req(scales, "scales", (scale_dtype,), shape=(N, G))
    _req(zeros, "zeros", (torch.uint8,), shape=(N, _zero_cols(G, bits)))
    return N, K


def _tokens(x: torch.Tensor, K: int, name: str, dtypes=_HALVES) -> torch.Tensor:
    """Activations [T, K] (a 1-D [K] vector is one token)."""
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    x2 = x.reshape(1, -1) if x.dim() == 1 else x
    _req(x2, name, dtypes, shape=(None, K))
    return x2


# ---------------------------------------------------------------------------
# Sizes.
# ---------------------------------------------------------------------------
def w4_sizes(N: int, K: int, group: int = GROUP) -> Tuple[int, int, int]:
    """(codes, scales, zeros) byte sizes of the INT4 format."""
    c, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _call("qmm_w4_sizes", N, K, group, ctypes.byref(c), ctypes.byref(s), ctypes.byref(z))
    return c.value, s.value, z.value


def wq_sizes(N: int, K: int, group: int = GROUP, bits: int = 4,
             scale_dtype: torch.dtype = torch.float32) -> Tuple[int, int, int]:
    """(codes, scales, zeros) byte sizes of any stored format."""
    c, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _call("qmm_wq_sizes", N, K, group, bits, _sdt(scale_dtype), ctypes.byref(c), ctypes.byref(s), ctypes.byref(z))
    return c.value, s.value, z.value


# ---------------------------------------------------------------------------
# Quantization and dequantization.
# ---------------------------------------------------------------------------
def _quant_outputs(W, group, bits, scale_dtype):
    _req(W, "W", _FLOATS, ndim=2)
    if bits not in (3, 4, 8):
        raise ValueError(f"bits must be 3, 4 or 8, not {bits}")
    N, K = W.shape
    G = _groups(K, group)
    dev = _place(W=W)
    codes = torch.empty((N, _code_cols(K, bits)), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, G), dtype=scale_dtype, device=dev)
    zeros = torch.empty((N, _zero_cols(G, bits)), dtype=torch.uint8, device=dev)
    return N, K, codes, scales, zeros


def quantize_groupwise_ex(W: torch.Tensor, group: int = GROUP, bits: int = 4,
                          scale_dtype: torch.dtype = torch.float32, symmetric: bool = False):
    """W [N, K] (fp32 / bf16 / fp16) -> (codes, scales, zeros) in a stored format:
    group 32..1024, 3, 4 or 8 bits, fp32 or fp16 scales, asymmetric or symmetric grid."""
    sdt = _sdt(scale_dtype)
    N, K, codes, scales, zeros = _quant_outputs(W, group, bits, scale_dtype)
    _call("quantize_groupwise_ex", _ptr(W), _dt(W.dtype), N, K, group, bits, sdt, int(symmetric),
          _ptr(codes), _ptr(scales), _ptr(zeros), _stream(W))
    return codes, scales, zeros


def quantize_groupwise(W: torch.Tensor, group: int = GROUP, bits: int = 4, symmetric: bool = False):
    """W [N, K] (fp32 / bf16 / fp16) -> codes u8 [N, K/2], scales f32 [N, G], zeros u8 [N, ceil(G/2)]
    (other group sizes / bit widths: the stored formats with fp32 scales).
    symmetric=True: the symmetric grid, stored with zero-point 2^(bits-1) in the same format."""
    N, K, codes, scales, zeros = _quant_outputs(W, group, bits, torch.float32)
    _call("quantize_groupwise_symmetric" if symmetric else "quantize_groupwise", _ptr(W), _dt(W.dtype), N, K, group,
          bits, _ptr(codes), _ptr(scales), _ptr(zeros), _stream(W))
    return codes, scales, zeros


def quantize_groupwise_symmetric(W: torch.Tensor, group: int = GROUP, bits: int = 4):
    """Symmetric per-group quantization in the asymmetric storage format (zero-point 2^(bits-1))."""
    return quantize_groupwise(W, group, bits, symmetric=True)


def _scale_dtype_of(scales) -> torch.dtype:
    if not isinstance(scales, torch.Tensor):
        raise ValueError("scales must be a torch.Tensor")
    _sdt(scales.dtype)
    return scales.dtype


def dequantize_ex(codes, scales, zeros, dtype: torch.dtype = torch.float32, group: int = GROUP, bits: int = 4,
                  out: Optional[torch.Tensor] = None):
    """Stored format -> W_hat [N, K] in dtype (the scales' dtype selects fp32 or fp16 scales)."""
    sdt = _scale_dtype_of(scales)
    N, K = _check_format(codes, scales, zeros, group, bits, sdt)
    if dtype not in _FLOATS:
        raise ValueError(f"unsupported output dtype {dtype}")
    _out(out, (N, K), dtype)
    dev = _place(codes=codes, scales=scales, zeros=zeros, out=out)
    out = _alloc(out, (N, K), dtype, dev)
    _call("dequantize_ex", _ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, bits, _sdt(sdt), _ptr(out), _dt(dtype),
          _stream(codes))
    return out


def dequantize(codes, scales, zeros, dtype: torch.dtype = torch.float32, group: int = GROUP, bits: int = 4,
               out: Optional[torch.Tensor] = None):
    """Stored format with fp32 scales -> W_hat [N, K] in dtype."""
    N, K = _check_format(codes, scales, zeros, group, bits, torch.float32)
    if dtype not in _FLOATS:
        raise ValueError(f"unsupported output dtype {dtype}")
    _out(out, (N, K), dtype)
    dev = _place(codes=codes, scales=scales, zeros=zeros, out=out)
    out = _alloc(out, (N, K), dtype, dev)
    _call("dequantize", _ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, bits, _ptr(out), _dt(dtype),
          _stream(codes))
    return out


# ---------------------------------------------------------------------------
# Weight-only matmuls.
# ---------------------------------------------------------------------------
def _mm_args(codes, scales, zeros, x, group, bits, sdt, out, out_dtype, max_tokens=None, name="x"):
    N, K = _check_format(codes, scales, zeros, group, bits, sdt)
    x2 = _tokens(x, K, name)
    T = x2.shape[0]
    if max_tokens is not None and not 1 <= T <= max_tokens:
        raise ValueError(f"takes 1 to {max_tokens} tokens, not {T}")
    odt = out.dtype if out is not None else (out_dtype or x2.dtype)
    _out(out, (T, N), odt)
    dev = _place(codes=codes, scales=scales, zeros=zeros, **{name: x2}, out=out)
    return N, K, T, x2, _alloc(out, (T, N), odt, dev)


def w4a16_gemv(codes, scales, zeros, x: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
               group: int = GROUP, out: Optional[torch.Tensor] = None):
    """y [B, N] = x [B, K] @ W_hat^T for B <= 8 (decode), INT4 codes with fp32 scales."""
    N, K, B, x2, out = _mm_args(codes, scales, zeros, x, group, 4, torch.float32, out, out_dtype, 8)
    _call("w4a16_gemv", _ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, _ptr(x2), _dt(x2.dtype), B, _ptr(out),
          _dt(out.dtype), _stream(x2))
    return out


def w4a16_gemm(codes, scales, zeros, X: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
               group: int = GROUP, out: Optional[torch.Tensor] = None):
    """Y [M, N] = X [M, K] @ W_hat^T (bf16 or fp16 activations, fp32 accumulation)."""
    N, K, M, X2, out = _mm_args(codes, scales, zeros, X, group, 4, torch.float32, out, out_dtype, None, "X")
    _call("w4a16_gemm", _ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, _ptr(X2), _dt(X2.dtype), M, _ptr(out),
          _dt(out.dtype), _stream(X2))
    return out


def wxa16_gemv(codes, scales, zeros, x: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
               group: int = GROUP, bits: int = 4, out: Optional[torch.Tensor] = None):
    """y [B, N] = x [B, K] @ W_hat^T for B <= 8 on any stored format (the scales' dtype selects fp32 / fp16)."""
    sdt = _scale_dtype_of(scales)
    N, K, B, x2, out = _mm_args(codes, scales, zeros, x, group, bits, sdt, out, out_dtype, 8)
    _call("wxa16_gemv", _ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, bits, _sdt(sdt), _ptr(x2), _dt(x2.dtype),
          B, _ptr(out), _dt(out.dtype), _stream(x2))
    return out


def wxa16_gemm(codes, scales, zeros, X: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
               group: int = GROUP, bits: int = 4, out: Optional[torch.Tensor] = None):
    """Y [M, N] = X [M, K] @ W_hat^T on any stored format."""
    sdt = _scale_dtype_of(scales)
    N, K, M, X2, out = _mm_args(codes, scales, zeros, X, group, bits, sdt, out, out_dtype, None, "X")
    _call("wxa16_gemm", _ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, bits, _sdt(sdt), _ptr(X2), _dt(X2.dtype),
          M, _ptr(out), _dt(out.dtype), _stream(X2))
    return out


def _repack(name, src, out, what):
    _req(src, what, (torch.uint8,), ndim=2)
    _out(out, tuple(src.shape), torch.uint8)
    dev = _place(**{what: src}, out=out)
    out = _alloc(out, tuple(src.shape), torch.uint8, dev)
    _call(name, _ptr(src), _ptr(out), src.shape[0], src.shape[1] * 2, _stream(src))
    return out


def w4_repack_from_plain(plain: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """4-bit codes [N, K/2] in plain nibble order -> the library's code words (same shape)."""
    return _repack("qmm_w4_repack_from_plain", plain, out, "plain")


def w4_repack_to_plain(codes: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The library's 4-bit code words [N, K/2] -> plain nibble order (same shape)."""
    return _repack("qmm_w4_repack_to_plain", codes, out, "codes")


def w8a16_gemv(qW, w_scale, x: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None):
    """y [B, N] = w_scale[n] * (x [B, K] @ qW^T) for B <= 8 (weight-only INT8 decode)."""
    _req(qW, "qW", (torch.int8,), ndim=2)
    N, K = qW.shape
    _req(w_scale, "w_scale", (torch.float32,), shape=(N,))
    x2 = _tokens(x, K, "x")
    B = x2.shape[0]
    if not 1 <= B <= 8:
        raise ValueError(f"w8a16_gemv takes 1 to 8 tokens, not {B}")
    odt = out.dtype if out is not None else (out_dtype or x2.dtype)
    _out(out, (B, N), odt)
    dev = _place(qW=qW, w_scale=w_scale, x=x2, out=out)
    out = _alloc(out, (B, N), odt, dev)
    _call("w8a16_gemv", _ptr(qW), _ptr(w_scale), N, K, _ptr(x2), _dt(x2.dtype), B, _ptr(out), _dt(out.dtype),
          _stream(x2))
    return out


# ---------------------------------------------------------------------------
# SmoothQuant W8A8.
# ---------------------------------------------------------------------------
def _smooth_arg(smooth, K: int) -> None:
    if smooth is not None:
        _req(smooth, "smooth", (torch.float32,), shape=(K,))


def sq_smooth_factors(X: torch.Tensor, W: torch.Tensor, alpha: float = 0.5):
    """-> (smooth [K], x_colmax [K], w_colmax [K]) float32."""
    _req(X, "X", _FLOATS, ndim=2)
    M, K = X.shape
    _req(W, "W", _FLOATS, shape=(None, K))
    N = W.shape[0]
    dev = _place(X=X, W=W)
    smooth = torch.empty(K, dtype=torch.float32, device=dev)
    cx = torch.empty_like(smooth)
    cw = torch.empty_like(smooth)
    _call("sq_smooth_factors", _ptr(X), _dt(X.dtype), M, _ptr(W), _dt(W.dtype), N, K, alpha, _ptr(cx), _ptr(cw),
          _ptr(smooth), _stream(X))
    return smooth, cx, cw


def sq_quantize_weight(W: torch.Tensor, smooth: Optional[torch.Tensor] = None):
    """-> (qW int8 [N, K], w_scale f32 [N])."""
    _req(W, "W", _FLOATS, ndim=2)
    N, K = W.shape
    _smooth_arg(smooth, K)
    dev = _place(W=W, smooth=smooth)
    q = torch.empty((N, K), dtype=torch.int8, device=dev)
    s = torch.empty(N, dtype=torch.float32, device=dev)
    _call("sq_quantize_weight", _ptr(W), _dt(W.dtype), _ptr(smooth), N, K, _ptr(q), _ptr(s), _stream(W))
    return q, s


def sq_quantize_activation(X: torch.Tensor, smooth: Optional[torch.Tensor] = None, per_tensor: bool = False):
    """-> (qX int8 [M, K], x_scale f32 [M]); per_tensor=True: one scale for the whole X, repeated per row."""
    _req(X, "X", _FLOATS, ndim=2)
    M, K = X.shape
    _smooth_arg(smooth, K)
    dev = _place(X=X, smooth=smooth)
    q = torch.empty((M, K), dtype=torch.int8, device=dev)
    s = torch.empty(M, dtype=torch.float32, device=dev)
    _call("sq_quantize_activation_per_tensor" if per_tensor else "sq_quantize_activation", _ptr(X), _dt(X.dtype),
          _ptr(smooth), M, K, _ptr(q), _ptr(s), _stream(X))
    return q, s


def sq_quantize_activation_per_tensor(X: torch.Tensor, smooth: Optional[torch.Tensor] = None):
    """-> (qX int8 [M, K], x_scale f32 [M]) with one scale for the whole X, repeated per row."""
    return sq_quantize_activation(X, smooth, per_tensor=True)


def sq_int8_gemm(qX, x_scale, qW, w_scale, out_dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None):
    """Y [M, N] = (qX qW^T) * x_scale[m] * w_scale[n]; out_dtype int32 returns the raw accumulator."""
    _req(qX, "qX", (torch.int8,), ndim=2)
    M, K = qX.shape
    _req(qW, "qW", (torch.int8,), shape=(None, K))
    N = qW.shape[0]
    odt = out.dtype if out is not None else out_dtype
    raw = odt == torch.int32
    if not raw:
        _req(x_scale, "x_scale", (torch.float32,), shape=(M,))
        _req(w_scale, "w_scale", (torch.float32,), shape=(N,))
    _out(out, (M, N), odt)
    dev = _place(qX=qX, qW=qW, x_scale=None if raw else x_scale, w_scale=None if raw else w_scale, out=out)
    out = _alloc(out, (M, N), odt, dev)
    _call("sq_int8_gemm", _ptr(qX), _ptr(x_scale), _ptr(qW), _ptr(w_scale), M, N, K, _ptr(out), _dt(out.dtype),
          _stream(qX))
    return out


def sq_workspace_bytes(M: int, K: int) -> int:
    return int(lib().sq_workspace_bytes(M, K))


def _online_args(X, smooth, qW, w_scale, out, out_dtype, workspace=None):
    _req(X, "X", _FLOATS, ndim=2)
    M, K = X.shape
    _smooth_arg(smooth, K)
    _req(qW, "qW", (torch.int8,), shape=(None, K))
    N = qW.shape[0]
    _req(w_scale, "w_scale", (torch.float32,), shape=(N,))
    odt = out.dtype if out is not None else out_dtype
    _out(out, (M, N), odt)
    if workspace is not None:
        _req(workspace, "workspace", (torch.uint8,), ndim=1)
        if workspace.numel() < sq_workspace_bytes(M, K):
            raise ValueError(f"workspace holds {workspace.numel()} bytes; {sq_workspace_bytes(M, K)} needed")
    dev = _place(X=X, smooth=smooth, qW=qW, w_scale=w_scale, out=out, workspace=workspace)
    return M, N, K, dev, _alloc(out, (M, N), odt, dev)


def smooth_quant_w8a8_gemm(X: torch.Tensor, smooth: Optional[torch.Tensor], qW, w_scale,
                           out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None):
    """Online W8A8 step: per-token smoothing + INT8 quantization of X, INT8 GEMM, rescale."""
    M, N, K, dev, out = _online_args(X, smooth, qW, w_scale, out, out_dtype, workspace)
    if workspace is None:
        workspace = torch.empty(sq_workspace_bytes(M, K), dtype=torch.uint8, device=dev)
    _call("smooth_quant_w8a8_gemm", _ptr(X), _dt(X.dtype), _ptr(smooth), _ptr(qW), _ptr(w_scale), M, N, K,
          _ptr(out), _dt(out.dtype), _ptr(workspace), workspace.numel(), _stream(X))
    return out


def smooth_quant_w8a8_gemm_noalloc(X: torch.Tensor, smooth: Optional[torch.Tensor], qW, w_scale,
                                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None):
    """smooth_quant_w8a8_gemm with the library's own device scratch instead of a
    workspace (for callers that cannot allocate; pass `out` to allocate nothing)."""
    M, N, K, dev, out = _online_args(X, smooth, qW, w_scale, out, out_dtype)
    _call("smooth_quant_w8a8_gemm_noalloc", _ptr(X), _dt(X.dtype), _ptr(smooth), _ptr(qW), _ptr(w_scale), M, N, K,
          _ptr(out), _dt(out.dtype), _stream(X))
    return out


# ---------------------------------------------------------------------------
# FP8 E4M3 W8A8 (codes are torch.uint8 holding OCP E4M3 bytes; view them as
# torch.float8_e4m3fn to read the values).
# ---------------------------------------------------------------------------
def fp8_quantize(X: torch.Tensor, per_tensor: bool = False):
    """-> (q uint8 [rows, K] E4M3 codes, scale f32 [rows]); s = max|x| / 448 per
    row, or one for the whole matrix (repeated per row) when per_tensor."""
    _req(X, "X", _FLOATS, ndim=2)
    rows, K = X.shape
    dev = _place(X=X)
    q = torch.empty((rows, K), dtype=torch.uint8, device=dev)
    s = torch.empty(rows, dtype=torch.float32, device=dev)
    _call("fp8_quantize", _ptr(X), _dt(X.dtype), rows, K, int(per_tensor), _ptr(q), _ptr(s), _stream(X))
    return q, s


def fp8_gemm(qX, x_scale, qW, w_scale, out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None):
    """Y [M, N] = (E4M3(qX) E4M3(qW)^T) * x_scale[m] * w_scale[n] (fp32 accumulation)."""
    _req(qX, "qX", (torch.uint8,), ndim=2)
    M, K = qX.shape
    _req(qW, "qW", (torch.uint8,), shape=(None, K))
    N = qW.shape[0]
    _req(x_scale, "x_scale", (torch.float32,), shape=(M,))
    _req(w_scale, "w_scale", (torch.float32,), shape=(N,))
    odt = out.dtype if out is not None else out_dtype
    _out(out, (M, N), odt)
    dev = _place(qX=qX, qW=qW, x_scale=x_scale, w_scale=w_scale, out=out)
    out = _alloc(out, (M, N), odt, dev)
    _call("fp8_gemm", _ptr(qX), _ptr(x_scale), _ptr(qW), _ptr(w_scale), M, N, K, _ptr(out), _dt(out.dtype),
          _stream(qX))
    return out


def fp8_w8a8_gemm(X: torch.Tensor, qW, w_scale, out_dtype: torch.dtype = torch.bfloat16,
                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Online FP8 step: per-token E4M3 quantization of X, then fp8_gemm."""
    _req(X, "X", _FLOATS, ndim=2)
    M, K = X.shape
    _req(qW, "qW", (torch.uint8,), shape=(None, K))
    N = qW.shape[0]
    _req(w_scale, "w_scale", (torch.float32,), shape=(N,))
    odt = out.dtype if out is not None else out_dtype
    _out(out, (M, N), odt)
    if workspace is not None:
        _req(workspace, "workspace", (torch.uint8,), ndim=1)
        if workspace.numel() < sq_workspace_bytes(M, K):
            raise ValueError(f"workspace holds {workspace.numel()} bytes; {sq_workspace_bytes(M, K)} needed")
    dev = _place(X=X, qW=qW, w_scale=w_scale, out=out, workspace=workspace)
    out = _alloc(out, (M, N), odt, dev)
    if workspace is None:
        workspace = torch.empty(sq_workspace_bytes(M, K), dtype=torch.uint8, device=dev)
    _call("fp8_w8a8_gemm", _ptr(X), _dt(X.dtype), _ptr(qW), _ptr(w_scale), M, N, K, _ptr(out), _dt(out.dtype),
          _ptr(workspace), workspace.numel(), _stream(X))
    return out


# ---------------------------------------------------------------------------
# LLM.int8(): vector-wise INT8 with the outlier feature dimensions multiplied
# in 16-bit.  qW / w_scale are the per-output-channel INT8 weights
# (sq_quantize_weight(W) with no smoothing).
# ---------------------------------------------------------------------------
def _llm_args(X, threshold, max_outliers):
    _req(X, "X", _HALVES, ndim=2)
    M, K = X.shape
    if not threshold >= 0.0:
        raise ValueError(f"threshold must be >= 0, not {threshold}")
    cap = K if max_outliers is None else int(max_outliers)
    if cap < 0:
        raise ValueError(f"max_outliers must be >= 0, not {max_outliers}")
    return M, K, min(cap, K)


def llm_int8_outliers(X: torch.Tensor, threshold: float = 6.0, max_outliers: Optional[int] = None):
    """Outlier detection: -> (factor f32 [K]: +inf for each carved-out column, 1
    otherwise; index int32 [kept] in increasing column order; found).  The
    first `max_outliers` (default K) outlier columns are carved out.
    Synchronizes with the device to read the counts."""
    M, K, cap = _llm_args(X, threshold, max_outliers)
    dev = _place(X=X)
    factor = torch.empty(K, dtype=torch.float32, device=dev)
    index = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    counts = torch.empty(2, dtype=torch.int32, device=dev)
    _call("llm_int8_outliers", _ptr(X), _dt(X.dtype), M, K, float(threshold), cap, _ptr(factor), _ptr(index),
          _ptr(counts), _stream(X))
    kept, found = (int(v) for v in counts.cpu())
    return factor, index[:kept], found


def llm_int8_workspace_bytes(M: int, N: int, K: int, max_outliers: Optional[int] = None) -> int:
    return int(lib().llm_int8_workspace_bytes(M, N, K, K if max_outliers is None else max_outliers))


def llm_int8_gemm(X: torch.Tensor, qW, w_scale, threshold: float = 6.0, max_outliers: Optional[int] = None,
                  out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, n_outliers: Optional[torch.Tensor] = None):
    """Y [M, N] = S_out (X_q qW^T) + X_16 W_16^T: per-token INT8 of the columns of X
    whose largest |x| stays below `threshold`, the others (at most `max_outliers`,
    default K) multiplied in 16-bit.  `n_outliers` (int32 [1], device, optional)
    receives the number of outlier columns found."""
    M, K, cap = _llm_args(X, threshold, max_outliers)
    _req(qW, "qW", (torch.int8,), shape=(None, K))
    N = qW.shape[0]
    _req(w_scale, "w_scale", (torch.float32,), shape=(N,))
    odt = out.dtype if out is not None else out_dtype
    if odt not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, not {odt}")
    _out(out, (M, N), odt)
    if n_outliers is not None:
        _req(n_outliers, "n_outliers", (torch.int32,), shape=(1,))
    need = llm_int8_workspace_bytes(M, N, K, cap)
    if workspace is not None:
        _req(workspace, "workspace", (torch.uint8,), ndim=1)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes; {need} needed")
    dev = _place(X=X, qW=qW, w_scale=w_scale, out=out, workspace=workspace, n_outliers=n_outliers)
    out = _alloc(out, (M, N), odt, dev)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _call("llm_int8_gemm", _ptr(X), _dt(X.dtype), _ptr(qW), _ptr(w_scale), M, N, K, float(threshold), cap,
          _ptr(out), _dt(out.dtype), _ptr(n_outliers), _ptr(workspace), workspace.numel(), _stream(X))
    return out


# ---------------------------------------------------------------------------
# AWQ scaling search.
# ---------------------------------------------------------------------------
# 0, 0.1, .., 1 as numpy's linspace(0, 1, 11) has them (i * 0.1, the last one
# exactly 1): the grid of the awq listing in "Quantization from Scratch"
AWQ_ALPHAS = tuple(i * 0.1 for i in range(10)) + (1.0,)


def awq_workspace_bytes(N: int, K: int, T: int, n_alpha: int) -> int:
    return int(lib().awq_workspace_bytes(N, K, T, n_alpha))


def awq_search(W: torch.Tensor, X: torch.Tensor, alphas: Sequence[float] = AWQ_ALPHAS,
               workspace: Optional[torch.Tensor] = None):
    """AWQ on 16-bit weights W [N, K] with calibration activations X [T, K] of
    the same type (bf16 or fp16): returns (codes, scales, zeros) of
    W diag(s_best) in the INT4 group-128 format, smooth [K] (= s_best), err
    fp64 [len(alphas)] and best (int64 [1]), all on the device."""
    _req(W, "W", _HALVES, ndim=2)
    N, K = W.shape
    _req(X, "X", (W.dtype,), shape=(None, K))
    T = X.shape[0]
    a = [float(v) for v in alphas]
    if not 1 <= len(a) <= 64:
        raise ValueError(f"takes 1 to 64 alphas, not {len(a)}")
    if not all(0.0 <= v <= 1.0 for v in a):
        raise ValueError(f"alphas must lie in [0, 1]: {a}")
    if K % GROUP != 0:
        raise ValueError(f"K={K} is not a multiple of {GROUP}")
    need = awq_workspace_bytes(N, K, T, len(a))
    if workspace is not None:
        _req(workspace, "workspace", (torch.uint8,), ndim=1)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes; {need} needed")
    dev = _place(W=W, X=X, workspace=workspace)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // GROUP), dtype=torch.float32, device=dev)
    zeros = torch.empty((N, (K // GROUP + 1) // 2), dtype=torch.uint8, device=dev)
    smooth = torch.empty(K, dtype=torch.float32, device=dev)
    err = torch.empty(len(a), dtype=torch.float64, device=dev)
    best = torch.empty(1, dtype=torch.int64, device=dev)
    host_alphas = (ctypes.c_double * len(a))(*a)
    _call("awq_search", _ptr(W), _dt(W.dtype), _ptr(X), _dt(X.dtype), N, K, T, ctypes.cast(host_alphas, ctypes.c_void_p),
          len(a), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(smooth), _ptr(err), _ptr(best), _ptr(workspace),
          workspace.numel(), _stream(X))
    return codes, scales, zeros, smooth, err, best


def stream_read(data: torch.Tensor) -> torch.Tensor:
    """Read every byte of a contiguous device tensor once (a plain streaming
    read, for measuring bandwidth); returns the XOR of its 32-bit words as a
    uint32-valued int32 tensor [1] on the device."""
    if not isinstance(data, torch.Tensor):
        raise ValueError("data must be a torch.Tensor")
    nbytes = data.numel() * data.element_size()
    if nbytes == 0 or nbytes % 16 != 0:
        raise ValueError(f"data must hold a positive multiple of 16 bytes, not {nbytes}")
    dev = _place(data=data)
    out = torch.empty(1, dtype=torch.int32, device=dev)
    _call("qmm_stream_read", _ptr(data), nbytes, _ptr(out), _stream(data))
    return out


# ---------------------------------------------------------------------------
# 4-bit paged key/value cache.  cache: uint8 [pages, kv_heads, page, D + 8 D/g]
# (its shape carries the page and group sizes; include/qmm.h states the layout
# of a record).
# ---------------------------------------------------------------------------
def kv4_page_bytes(kv_heads: int, head_dim: int, page: int = 64, group: int = 64) -> int:
    """Bytes of one page of all heads; 0 for a shape that is not supported."""
    return int(lib().kv4_page_bytes(kv_heads, head_dim, page, group))


def kv4_cache(pages: int, kv_heads: int, head_dim: int, page: int = 64, group: int = 64, layers: Optional[int] = None,
              device="cuda") -> torch.Tensor:
    """An uninitialized cache, uint8 [pages, kv_heads, page, D + 8 D/g] (with `layers`: one such for each layer)."""
    if not kv4_page_bytes(kv_heads, head_dim, page, group):
        raise ValueError(f"unsupported cache shape: kv_heads={kv_heads} head_dim={head_dim} page={page} group={group}")
    shape = (pages, kv_heads, page, head_dim + 8 * (head_dim // group))
    return torch.empty(shape if layers is None else (layers, *shape), dtype=torch.uint8, device=device)


# Small calls are bound by what happens before the launch, so each operand is
# first compared with what is wanted in one expression, and only where that
# fails goes through the checks that name the fault.
def _cache_shape(cache, head_dim: int):
    """(pages, kv_heads, page, group) of a cache for heads of head_dim channels."""
    if type(cache) is not torch.Tensor or cache.dtype is not torch.uint8 or cache.dim() != 4:
        _req(cache, "cache", (torch.uint8,), ndim=4)
    pages, heads, page, token = cache.shape
    groups, rest = divmod(token - head_dim, 8)
    if groups <= 0 or rest or head_dim % groups:
        raise ValueError(f"cache has shape {tuple(cache.shape)}; a token of head_dim {head_dim} takes head_dim + 8 bytes "
                         "per group of channels")
    return pages, heads, page, head_dim // groups


def _rows(t, name: str, dtypes) -> Tuple:
    """Shape of rows of heads [T, heads, D]."""
    if type(t) is not torch.Tensor or t.dtype not in dtypes or t.dim() != 3:
        _req(t, name, dtypes, ndim=3)
    return t.shape


def _strides(t, name: str):
    """Token and head strides of rows of heads (strided views, as slices of a projection's output, are fine)."""
    ts, hs, cs = t.stride()
    if cs != 1 or (ts | hs) & 7:
        T, heads, D = t.shape                              # a single row's stride means nothing
        ts, hs = ts if T > 1 else 0, hs if heads > 1 else 0
        if cs != 1 and D > 1:
            raise ValueError(f"{name} must have its channels consecutive, has strides {t.stride()}")
        if (ts | hs) & 7:
            raise ValueError(f"{name} must have token and head strides that are multiples of 8, has strides {t.stride()}")
    return ts, hs


def _fresh(t: torch.Tensor, shape) -> torch.Tensor:
    """A dense tensor of t's shape and type (empty_like is half of new_empty's time, but keeps strides)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(shape)


def _vector(t, name: str, dtype, n: int) -> None:
    if type(t) is not torch.Tensor or t.dtype is not dtype or t.shape != (n,):
        _req(t, name, (dtype,), shape=(n,))


def _on(dev: int, strided: Sequence, **dense) -> None:
    """All operands on GPU `dev` (None entries are skipped), the dense ones contiguous."""
    if dev < 0:
        raise ValueError("the operands must be device tensors")
    for t in strided:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"an operand is on {t.device}, another on GPU {dev}")
    for name, t in dense.items():
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            if t.get_device() != dev:
                raise ValueError(f"{name} is on {t.device}, another operand on GPU {dev}")
            raise ValueError(f"{name} must be contiguous")


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor) -> None:
    """Quantize keys and values [T, kv_heads, D] into the slots (int64 [T], page id * page + place; distinct; -1
    writes nothing) of the cache."""
    T, heads, D = shape = _rows(k, "k", _HALVES)
    pages, kv_heads, page, group = _cache_shape(cache, D)
    if heads != kv_heads:
        raise ValueError(f"k has {heads} heads, the cache {kv_heads}")
    dtype = k.dtype
    if _rows(v, "v", (dtype,)) != shape:
        _req(v, "v", (dtype,), shape=shape)
    kt, kh = _strides(k, "k")
    vt, vh = _strides(v, "v")
    _vector(slots, "slots", torch.int64, T)
    _on(cache.get_device(), (k, v), cache=cache, slots=slots)
    _call_block("kv4_append", k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _DT[dtype], T, slots.data_ptr(),
                cache.data_ptr(), pages, heads, D, page, group, _stream(cache))


def kv4_read(cache: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype = torch.bfloat16):
    """-> (k, v) [T, kv_heads, head_dim] in dtype: the values that the codes of the slots (int64 [T]) stand for, zeros
    for a slot outside the cache."""
    if dtype not in _FLOATS:
        raise ValueError(f"unsupported output dtype {dtype}")
    pages, heads, page, group = _cache_shape(cache, head_dim)
    _req(slots, "slots", (torch.int64,), ndim=1)
    T = slots.shape[0]
    _on(cache.get_device(), (), cache=cache, slots=slots)
    k = cache.new_empty((T, heads, head_dim), dtype=dtype)
    v = torch.empty_like(k)
    _call_block("kv4_read", cache.data_ptr(), pages, heads, head_dim, page, group, slots.data_ptr(), T, k.data_ptr(),
                v.data_ptr(), _DT[dtype], _stream(cache))
    return k, v


def kv4_copy_pages(cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Copy page src[i] to page dst[i] (int64 [n]) in every layer of cache [layers, pages, kv_heads, page, token]
    (or of one layer's [pages, kv_heads, page, token]).  Destinations are distinct and no sources."""
    if not isinstance(cache, torch.Tensor) or cache.dim() not in (4, 5):
        raise ValueError("cache must be a torch.Tensor of 4 dimensions, or 5 with layers")
    _req(cache, "cache", (torch.uint8,))
    _req(src, "src", (torch.int64,), ndim=1)
    n = src.shape[0]
    _vector(dst, "dst", torch.int64, n)
    _on(cache.get_device(), (), cache=cache, src=src, dst=dst)
    *layers, pages, heads, page, token = cache.shape
    _call_block("kv4_copy_pages", cache.data_ptr(), layers[0] if layers else 1, pages, heads * page * token,
                src.data_ptr(), dst.data_ptr(), n, _stream(cache))


@functools.lru_cache(maxsize=4096)      # of sizes alone
def kv4_attention_workspace_bytes(T: int, seqs: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int,
                                  group: int, max_context: int, window: int = 0, sinks: int = 0) -> int:
    """Bytes that kv4_attention needs for these sizes (max_context: the page table's width in tokens); often 0."""
    return int(lib().kv4_attention_workspace_bytes(T, seqs, max_q, q_heads, kv_heads, head_dim, group, max_context,
                                                   window, sinks))


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, context: torch.Tensor,
                  cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None, scale: Optional[float] = None,
                  window: int = 0, sinks: int = 0, return_lse: bool = False, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None):
    """Causal attention of q [T, q_heads, D] over the cache: sequence b's context[b] (int32 [seqs]) tokens lie in the
    pages page_table[b] (int32 [seqs, width], -1 for pages that are gone), its queries are its last tokens, one each or
    rows cu_q[b] .. cu_q[b + 1] - 1 of q (int32 [seqs + 1]; max_q, a hint, the most of a sequence).  window: the keys a
    query sees (0: all before it), sinks: the first keys that stay visible.  Returns out [T, q_heads, D], with
    return_lse also the fp32 log-sum-exp [T, q_heads]; a row that sees no key is 0 and -inf."""
    T, q_heads, D = shape = _rows(q, "q", _HALVES)
    dtype = q.dtype
    pages, kv_heads, page, group = _cache_shape(cache, D)
    if q_heads % kv_heads:
        raise ValueError(f"q has {q_heads} heads, not a multiple of the cache's {kv_heads}")
    qt, qh = _strides(q, "q")
    if type(page_table) is not torch.Tensor or page_table.dtype is not torch.int32 or page_table.dim() != 2:
        _req(page_table, "page_table", (torch.int32,), ndim=2)
    seqs, width = page_table.shape
    _vector(context, "context", torch.int32, seqs)
    stride, one = page_table.stride()
    if width > 1 and one != 1:
        raise ValueError(f"page_table must have consecutive rows, has strides {page_table.stride()}")
    if seqs < 2:
        stride = width
    if cu_q is not None:
        _vector(cu_q, "cu_q", torch.int32, seqs + 1)
        most = max(1, T if max_q is None else int(max_q))
    elif T != seqs:
        raise ValueError(f"q has {T} rows for {seqs} sequences: without cu_q each has one")
    else:
        most = 1
    if window < 0 or sinks < 0:
        raise ValueError(f"window and sinks must be >= 0, not {window} and {sinks}")
    if out is not None:
        _out(out, shape, dtype)
    _on(q.get_device(), (page_table,), cache=cache, context=context, cu_q=cu_q, out=out, workspace=workspace)
    need = kv4_attention_workspace_bytes(T, seqs, most, q_heads, kv_heads, D, group, width * page, window, sinks)
    if workspace is not None:
        _req(workspace, "workspace", (torch.uint8,), ndim=1)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes; {need} needed")
    elif need:
        workspace = cache.new_empty(need)
    if out is None:
        out = _fresh(q, shape)
    lse = q.new_empty((T, q_heads), dtype=torch.float32) if return_lse else None
    _call_block("kv4_attention", q.data_ptr(), qt, qh, _DT[dtype], T, q_heads, _ptr0(cu_q), seqs, most,
                context.data_ptr(), page_table.data_ptr(), width, stride, cache.data_ptr(), pages, kv_heads, D, page,
                group, D ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), _ptr0(lse), _ptr0(workspace),
                need if workspace is not None else 0, _stream(q))
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------------------
# Norms of queries and keys with the rotation by position.
# ---------------------------------------------------------------------------
def rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original: int = 4096, low: float = 1.0, high: Optional[float] = None):
    """-> (frequencies [rot/2] in radians per position, magnitude) for `rot` rotated channels, base^(-2i/rot), scaled
    for contexts `factor` times the `original` one:
      "linear"      every frequency over factor (positions interpolated);
      "ntk"         the base raised by factor^(rot / (rot - 2)), so the slowest pair is interpolated, the fastest kept;
      "wavelength"  a pair that turns more than `high` (default 4) times in the original context keeps its frequency,
                    one that turns less than `low` times is divided by factor, linear in the turns between;
      "yarn"        the same two ends (high default 32), linear in the pair's index between (where every pair turns
                    more than `low` times, the ramp goes on past the last one), and the rotated channels grow by
                    0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and positive, not {rot}")
    if base <= 0 or factor <= 0:
        raise ValueError(f"base and factor must be positive, not {base} and {factor}")
    half = rot // 2
    f = [base ** (-i / half) for i in range(half)]
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot >= 4")
        raised = base * factor ** (rot / (rot - 2))
        return [raised ** (-i / half) for i in range(half)], 1.0
    if scaling not in ("wavelength", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    high = (4.0 if scaling == "wavelength" else 32.0) if high is None else high
    if not 0 < low < high:
        raise ValueError(f"needs 0 < low < high, not {low} and {high}")
    if scaling == "wavelength":
        keep = [min(1.0, max(0.0, (original * v / (2 * math.pi) - low) / (high - low))) for v in f]
        return [k * v + (1.0 - k) * v / factor for k, v in zip(keep, f)], 1.0
    index = lambda turns: half * math.log(original / (2 * math.pi * turns)) / math.log(base)
    first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
    keep = [1.0 - min(1.0, max(0.0, (i - first) / max(last - first, 0.001))) for i in range(half)]
    return [k * v + (1.0 - k) * v / factor for k, v in zip(keep, f)], \
        0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def rope_table(rows: int, frequencies: Sequence[float], magnitude: float = 1.0, device="cuda") -> torch.Tensor:
    """float32 [rows, len(frequencies), 2] of cosines and sines of position * frequency (times magnitude), for
    positions 0 .. rows - 1; computed in fp64."""
    half = len(frequencies)
    if not 1 <= half <= 256 or rows < 1:
        raise ValueError(f"takes 1 to 256 frequencies and at least one row, not {half} and {rows}")
    table = torch.empty((rows, half, 2), dtype=torch.float32, device=device)
    _place(table=table)
    host = (ctypes.c_double * half)(*[float(v) for v in frequencies])
    _call("rope_table", ctypes.cast(host, ctypes.c_void_p), half, rows, float(magnitude), _ptr(table), _stream(table))
    return table


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor] = None,
                 table: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Norms of each head of q [T, q_heads, D] and k [T, k_heads, D] (RMS, where its weight [D] is given, in their type
    or fp32) and the rotation of its first 2 * table.shape[1] channels at positions (int64 [T]) by the table, in halves
    or interleaved pairs; returns (q_out, k_out).  k may be None, q_out / k_out the inputs themselves (dense ones)."""
    T, q_heads, D = shape = _rows(q, "q", _HALVES)
    dtype = q.dtype
    qt, qh = _strides(q, "q")
    k_heads = kt = kh = 0
    if k is not None:
        k_shape = _rows(k, "k", (dtype,))
        k_heads = k_shape[1]
        if k_shape != (T, k_heads, D):
            _req(k, "k", (dtype,), shape=(T, None, D))
        kt, kh = _strides(k, "k")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    if q_out is not None or k_out is not None:
        _out(q_out, shape, dtype, "q_out")
        _out(k_out, (T, k_heads, D), dtype, "k_out")
    w_dtype = dtype
    if q_weight is not None:
        w_dtype = torch.float32 if q_weight.dtype is torch.float32 else dtype
        _vector(q_weight, "q_weight", w_dtype, D)
    if k_weight is not None:
        if q_weight is None and k_weight.dtype is torch.float32:
            w_dtype = torch.float32
        _vector(k_weight, "k_weight", w_dtype, D)
    if not eps >= 0.0:
        raise ValueError(f"eps must be >= 0, not {eps}")
    rows = rot = 0
    if table is not None:
        if type(table) is not torch.Tensor or table.dtype is not torch.float32 or table.dim() != 3 or table.shape[2] != 2:
            _req(table, "table", (torch.float32,), shape=(None, None, 2))
        rows, half, _ = table.shape
        rot = 2 * half
        if rot > D:
            raise ValueError(f"table rotates {rot} channels of heads of {D}")
        _vector(positions, "positions", torch.int64, T)
    elif positions is not None:
        raise ValueError("positions need a table")
    _on(q.get_device(), (k,), q_weight=q_weight, k_weight=k_weight, positions=positions, table=table, q_out=q_out,
        k_out=k_out)
    if q_out is None:
        q_out = _fresh(q, shape)
    if k is not None and k_out is None:
        k_out = _fresh(k, k_shape)
    _call_block("qk_norm_rope", q.data_ptr(), qt, qh, q_heads, _ptr0(k), kt, kh, k_heads, _DT[dtype], T, D,
                _ptr0(positions), _ptr0(table), rows, rot, interleaved, _ptr0(q_weight), _ptr0(k_weight), _DT[w_dtype],
                eps, q_out.data_ptr(), _ptr0(k_out), _stream(q))
    return q_out, k_out
