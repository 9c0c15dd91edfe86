"""ctypes binding of libgptq_mi355x.so (argument marshalling only).

Every computation happens in the library's HIP kernels; this module converts
torch tensors into device pointers, passes the current HIP stream and maps a
non-zero status to an exception.  It never computes a result itself, and it
fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgptq_mi355x.so")

GPTQ_OK = 0
GPTQ_ERR_INVALID_ARG = 1
GPTQ_ERR_NOT_PD = 2
GPTQ_ERR_NONFINITE = 3
GPTQ_ERR_EMPTY = 4
GPTQ_ERR_WORKSPACE = 5
GPTQ_ERR_HIP = 6
GPTQ_ERR_UNSUPPORTED = 7

GPTQ_F32 = 0
GPTQ_BF16 = 1

# every symbol the C header declares
EXPORTED = (
    "gptq_abi_version",
    "gptq_status_str",
    "gptq_hessian_workspace_size",
    "gptq_hessian_accumulate",
    "gptq_prepare_workspace_size",
    "gptq_prepare",
    "gptq_quantize_workspace_size",
    "gptq_quantize_layer",
    "gptq_quantize_layer_noalloc",
    "gptq_pack",
    "gptq_pack_ordered",
    "gptq_dequant_gemm_workspace_size",
    "gptq_dequant_gemm",
    "gptq_gather_columns",
    "gptq_dequantize",
    "gptq_gemm_bf16",
    "gptq_swiglu",
    "gptq_residual_add",
    "awq_absum_workspace_size",
    "awq_activation_absum",
    "awq_lite_workspace_size",
    "awq_lite",
    "awq_clip_quantize",
    "rtn_minmax",
    "gptq_layer_error_workspace_size",
    "gptq_layer_error",
    "fp8_quantize_rows",
    "fp8_swiglu_quantize",
    "fp8_quantize_blocks",
    "fp8_gemm_workspace_size",
    "fp8_gemm",
    "fp8_linear_workspace_size",
    "fp8_linear",
    "fp8_gated_gemm_workspace_size",
    "fp8_gated_gemm",
    "kv_cache_write_workspace_size",
    "kv_cache_write",
    "kv_cache_read",
    "token_logprobs_workspace_size",
    "token_logprobs",
)

FP8_BLOCK = 128  # columns (and weight rows) that share a scale
GPTQ_KV_INT4 = 0
GPTQ_KV_INT8 = 1
GPTQ_KV_E4M3 = 2
GPTQ_KV_SMALL_TOKENS = 1024  # kv_cache_write needs no workspace up to here
_KV_FORMATS = {"int4": GPTQ_KV_INT4, "int8": GPTQ_KV_INT8, "e4m3": GPTQ_KV_E4M3}


class GPTQConfig(ctypes.Structure):
    _fields_ = [
        ("bits", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("perc_damp", ctypes.c_float),
        ("desc_act", ctypes.c_int32),
        ("sym", ctypes.c_int32),
        ("static_groups", ctypes.c_int32),
    ]


class GPTQKVCache(ctypes.Structure):
    """A quantized paged cache of keys or values (make_kv_cache builds one); it
    keeps its tensors alive and may be kept for as long as they are in use."""

    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("zeros", ctypes.c_void_p),
        ("pages", ctypes.c_int64),
        ("page_stride", ctypes.c_int64),
        ("slot_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("param_page_stride", ctypes.c_int64),
        ("param_slot_stride", ctypes.c_int64),
        ("param_head_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("format", ctypes.c_int32),
    ]


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t


def load() -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python post_weight_quantization_22_amd/build.py` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    lib.gptq_abi_version.restype = ctypes.c_uint32
    lib.gptq_abi_version.argtypes = []
    lib.gptq_status_str.restype = ctypes.c_char_p
    lib.gptq_status_str.argtypes = [_i32]
    lib.gptq_hessian_workspace_size.restype = _i32
    lib.gptq_hessian_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(_sz)]
    lib.gptq_hessian_accumulate.restype = _i32
    lib.gptq_hessian_accumulate.argtypes = [_vp, _i64, _i64, _vp, _i32, _i64, _i64, _vp, _sz, _vp]
    lib.gptq_prepare_workspace_size.restype = _i32
    lib.gptq_prepare_workspace_size.argtypes = [_i64, ctypes.POINTER(_sz)]
    lib.gptq_prepare.restype = _i32
    lib.gptq_prepare.argtypes = [_vp, _i64, _i64, _i64, ctypes.c_float, _i32, _vp, _i64, _vp, _vp,
                                 _vp, _vp, _vp, _sz, _vp]
    lib.gptq_quantize_workspace_size.restype = _i32
    lib.gptq_quantize_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(GPTQConfig),
                                                 ctypes.POINTER(_sz)]
    lib.gptq_quantize_layer.restype = _i32
    lib.gptq_quantize_layer.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _vp,
                                        ctypes.POINTER(GPTQConfig), _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _sz, _vp]
    lib.gptq_quantize_layer_noalloc.restype = _i32
    lib.gptq_quantize_layer_noalloc.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _vp,
                                                ctypes.POINTER(GPTQConfig), _vp, _vp, _vp, _vp,
                                                _vp, _vp, _vp]
    lib.gptq_pack.restype = _i32
    lib.gptq_pack.argtypes = [_vp, _i64, _i64, _i32, _vp, _vp]
    lib.gptq_pack_ordered.restype = _i32
    lib.gptq_pack_ordered.argtypes = [_vp, _i64, _i64, _i32, _vp, _vp, _vp]
    lib.gptq_dequant_gemm_workspace_size.restype = _i32
    lib.gptq_dequant_gemm_workspace_size.argtypes = [_i64, _i64, _i64, _i32, ctypes.POINTER(_sz)]
    lib.gptq_dequant_gemm.restype = _i32
    lib.gptq_dequant_gemm.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _i32, _i32, _vp,
                                      _vp, _vp, _i64, _vp, _i32, _i64, _vp, _sz, _vp]
    lib.gptq_dequantize.restype = _i32
    lib.gptq_dequantize.argtypes = [_vp, _i64, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp]
    lib.gptq_gemm_bf16.restype = _i32
    lib.gptq_gemm_bf16.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i32, _i64, _vp]
    lib.gptq_gather_columns.restype = _i32
    lib.gptq_gather_columns.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _vp]
    lib.gptq_swiglu.restype = _i32
    lib.gptq_swiglu.argtypes = [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp]
    lib.gptq_residual_add.restype = _i32
    lib.gptq_residual_add.argtypes = [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp]
    lib.awq_absum_workspace_size.restype = _i32
    lib.awq_absum_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(_sz)]
    lib.awq_activation_absum.restype = _i32
    lib.awq_activation_absum.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _sz, _vp]
    lib.awq_lite_workspace_size.restype = _i32
    lib.awq_lite_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(_sz)]
    lib.awq_lite.restype = _i32
    lib.awq_lite.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _i32, _i32,
                             _i32, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.awq_clip_quantize.restype = _i32
    lib.awq_clip_quantize.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i32, _i32,
                                      _i32, _i32, _vp, _vp, _vp, _vp, _vp]
    lib.rtn_minmax.restype = _i32
    lib.rtn_minmax.argtypes = [_vp, _i32, _i64, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp]
    lib.gptq_layer_error_workspace_size.restype = _i32
    lib.gptq_layer_error_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(_sz)]
    lib.gptq_layer_error.restype = _i32
    lib.gptq_layer_error.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp,
                                     _i64, _vp, _vp, _sz, _vp]
    lib.fp8_quantize_rows.restype = _i32
    lib.fp8_quantize_rows.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]
    lib.fp8_swiglu_quantize.restype = _i32
    lib.fp8_swiglu_quantize.argtypes = [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp,
                                        _i64, _vp]
    lib.fp8_quantize_blocks.restype = _i32
    lib.fp8_quantize_blocks.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]
    for name in ("fp8_gemm_workspace_size", "fp8_linear_workspace_size",
                 "fp8_gated_gemm_workspace_size"):
        getattr(lib, name).restype = _i32
        getattr(lib, name).argtypes = [_i64, _i64, _i64, ctypes.POINTER(_sz)]
    lib.fp8_gemm.restype = _i32
    lib.fp8_gemm.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp,
                             _i64, _vp, _i32, _i64, _vp, _sz, _vp]
    lib.fp8_linear.restype = _i32
    lib.fp8_linear.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i32,
                               _i64, _vp, _sz, _vp]
    lib.fp8_gated_gemm.restype = _i32
    lib.fp8_gated_gemm.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64,
                                   _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _sz, _vp]
    _kvp = _vp  # the address of a GPTQKVCache
    lib.kv_cache_write_workspace_size.restype = _i32
    lib.kv_cache_write_workspace_size.argtypes = [_i64, _kvp, ctypes.POINTER(_sz)]
    lib.kv_cache_write.restype = _i32
    lib.kv_cache_write.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _vp, _kvp, _kvp,
                                   _vp, _vp, _sz, _vp]
    lib.kv_cache_read.restype = _i32
    lib.kv_cache_read.argtypes = [_kvp, _kvp, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i32,
                                  _vp, _vp]
    lib.token_logprobs_workspace_size.restype = _i32
    lib.token_logprobs_workspace_size.argtypes = [_i64, _i64, _i32, ctypes.POINTER(_sz)]
    lib.token_logprobs.restype = _i32
    lib.token_logprobs.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _vp, _vp,
                                   _sz, _vp]
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().gptq_status_str(status).decode()


def _check(status: int, where: str) -> None:
    if status != GPTQ_OK:
        raise GPTQError(status, where, status_str(status))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return GPTQ_BF16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ld(t) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return t.stride(0)


def _workspace(nbytes: int, device, stream=None):
    """A per-call workspace allocated on the stream the call is enqueued on, so
    that torch's caching allocator does not hand the memory to other work
    before the library's kernels on that stream are done with it."""
    import torch

    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


_INT32_LIKE = ("int32", "uint32")


def _buf(t, name: str, shape, dtypes, device, optional: bool = True, min_rows=None):
    """Check an output or index buffer before its pointer goes to the library:
    the kernels write ``shape`` elements with the row stride the ABI states, so
    a smaller, strided, mistyped or foreign-device tensor would be written out
    of bounds.  ``shape`` entries of None are not checked; ``dtypes`` are torch
    dtype names."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if str(t.dtype).replace("torch.", "") not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if len(shape) == 1:
        if t.numel() < shape[0]:
            raise ValueError(f"{name}: {t.numel()} elements, need {shape[0]}")
        return
    if t.dim() != len(shape) or any(s is not None and d != s for d, s in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _mat(t, name: str, rows: int, cols: int, dtypes, device):
    """A 2-D operand read or written with an explicit row stride: unit column
    stride, at least ``rows`` x ``cols``, on ``device``."""
    if t is None:
        raise ValueError(f"{name} is required")
    if str(t.dtype).replace("torch.", "") not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 2 or t.stride(1) != 1 or t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"{name}: expected a 2-D tensor of at least {rows} x {cols} with unit "
                         f"column stride, got shape {tuple(t.shape)} strides {t.stride()}")


def _ngroups(n: int, group_size: int) -> int:
    return 1 if group_size <= 0 else -(-n // group_size)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def gptq_abi_version() -> int:
    return int(load().gptq_abi_version())


def gptq_status_str(status: int) -> str:
    return status_str(status)


def gptq_hessian_workspace_size(n: int, tokens: int) -> int:
    out = _sz(0)
    _check(load().gptq_hessian_workspace_size(n, tokens, ctypes.byref(out)),
           "gptq_hessian_workspace_size")
    return out.value


def gptq_hessian_accumulate(S, X, ws=None, stream=None) -> None:
    """S[n, n] (fp32, lower triangle) += X^T X for X[tokens, n] (bf16 or fp32)."""
    n = S.shape[0]
    tokens = X.shape[0]
    _mat(S, "S", n, n, ("float32",), S.device)
    _mat(X, "X", tokens, n, ("bfloat16", "float32"), S.device)
    need = gptq_hessian_workspace_size(n, tokens) if _dtype_code(X) == GPTQ_BF16 else 0
    if ws is None:
        ws = _workspace(need, S.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().gptq_hessian_accumulate(_ptr(S), n, _ld(S), _ptr(X), _dtype_code(X), tokens,
                                          _ld(X), _ptr(ws), nbytes, _stream(stream)),
           "gptq_hessian_accumulate")


def gptq_prepare_workspace_size(n: int) -> int:
    out = _sz(0)
    _check(load().gptq_prepare_workspace_size(n, ctypes.byref(out)), "gptq_prepare_workspace_size")
    return out.value


def gptq_prepare(S, tokens: int, perc_damp: float, desc_act: bool, U, perm=None, dead=None,
                 lambda_out=None, info=None, ws=None, stream=None) -> None:
    n = S.shape[0]
    d = S.device
    _mat(S, "S", n, n, ("float32",), d)
    _mat(U, "U", n, n, ("float32",), d)
    _buf(perm, "perm", (n,), _INT32_LIKE, d)
    _buf(dead, "dead", (n,), ("uint8", "bool"), d)
    _buf(lambda_out, "lambda_out", (1,), ("float32",), d)
    _buf(info, "info", (1,), ("int32",), d, optional=False)
    if ws is None:
        ws = _workspace(gptq_prepare_workspace_size(n), S.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().gptq_prepare(_ptr(S), n, _ld(S), int(tokens), float(perc_damp), int(desc_act),
                               _ptr(U), _ld(U), _ptr(perm), _ptr(dead), _ptr(lambda_out),
                               _ptr(info), _ptr(ws), nbytes, _stream(stream)),
           "gptq_prepare")


def make_config(bits: int, group_size: int, block_size: int = 128, perc_damp: float = 0.01,
                desc_act: bool = False, sym: bool = False,
                static_groups: bool = False) -> GPTQConfig:
    return GPTQConfig(bits, group_size, block_size, perc_damp, int(desc_act), int(sym),
                      int(static_groups))


def gptq_quantize_workspace_size(m: int, n: int, cfg: GPTQConfig) -> int:
    out = _sz(0)
    _check(load().gptq_quantize_workspace_size(m, n, ctypes.byref(cfg), ctypes.byref(out)),
           "gptq_quantize_workspace_size")
    return out.value


def gptq_quantize_layer(W, U, cfg: GPTQConfig, codes, scales, zeros, perm=None, dead=None,
                        g_idx=None, row_err=None, info=None, ws=None, stream=None) -> None:
    m, n = W.shape
    d = W.device
    ng = _ngroups(n, cfg.group_size)
    _mat(W, "W", m, n, ("bfloat16", "float32"), d)
    _mat(U, "U", n, n, ("float32",), d)
    _buf(codes, "codes", (m, n), ("uint8",), d, optional=False)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _buf(perm, "perm", (n,), _INT32_LIKE, d)
    _buf(dead, "dead", (n,), ("uint8", "bool"), d)
    _buf(g_idx, "g_idx", (n,), _INT32_LIKE, d)
    _buf(row_err, "row_err", (m,), ("float32",), d)
    _buf(info, "info", (1,), ("int32",), d)
    if ws is None:
        ws = _workspace(gptq_quantize_workspace_size(m, n, cfg), W.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().gptq_quantize_layer(_ptr(W), _dtype_code(W), m, n, _ld(W), _ptr(U), _ld(U),
                                      _ptr(perm), _ptr(dead), ctypes.byref(cfg), _ptr(codes),
                                      _ptr(scales), _ptr(zeros), _ptr(g_idx), _ptr(row_err),
                                      _ptr(info), _ptr(ws), nbytes, _stream(stream)),
           "gptq_quantize_layer")


GPTQ_NOALLOC_SCRATCH_BYTES = 64 << 20


def gptq_quantize_layer_noalloc(W, U, cfg: GPTQConfig, codes, scales, zeros, perm=None,
                                dead=None, g_idx=None, row_err=None, info=None,
                                stream=None) -> None:
    """gptq_quantize_layer on the library's fixed per-GPU scratch: allocates
    nothing (GPTQ_ERR_WORKSPACE for layers whose workspace exceeds it)."""
    m, n = W.shape
    d = W.device
    ng = _ngroups(n, cfg.group_size)
    _mat(W, "W", m, n, ("bfloat16", "float32"), d)
    _mat(U, "U", n, n, ("float32",), d)
    _buf(codes, "codes", (m, n), ("uint8",), d, optional=False)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _buf(perm, "perm", (n,), _INT32_LIKE, d)
    _buf(dead, "dead", (n,), ("uint8", "bool"), d)
    _buf(g_idx, "g_idx", (n,), _INT32_LIKE, d)
    _buf(row_err, "row_err", (m,), ("float32",), d)
    _buf(info, "info", (1,), ("int32",), d)
    _check(load().gptq_quantize_layer_noalloc(_ptr(W), _dtype_code(W), m, n, _ld(W), _ptr(U),
                                              _ld(U), _ptr(perm), _ptr(dead), ctypes.byref(cfg),
                                              _ptr(codes), _ptr(scales), _ptr(zeros),
                                              _ptr(g_idx), _ptr(row_err), _ptr(info),
                                              _stream(stream)),
           "gptq_quantize_layer_noalloc")


def gptq_pack(codes, bits: int, packed, stream=None) -> None:
    m, n = codes.shape
    _buf(codes, "codes", (m, n), ("uint8",), codes.device, optional=False)
    _buf(packed, "packed", (m, -(-(n * int(bits)) // 32)), _INT32_LIKE, codes.device,
         optional=False)
    _check(load().gptq_pack(_ptr(codes), m, n, int(bits), _ptr(packed), _stream(stream)),
           "gptq_pack")


def gptq_pack_ordered(codes, bits: int, perm, packed, stream=None) -> None:
    """packed[r] = codes[r, perm[0]], codes[r, perm[1]], ... in the gptq_pack layout."""
    m, n = codes.shape
    _buf(codes, "codes", (m, n), ("uint8",), codes.device, optional=False)
    _buf(perm, "perm", (n,), _INT32_LIKE, codes.device)
    _buf(packed, "packed", (m, -(-(n * int(bits)) // 32)), _INT32_LIKE, codes.device,
         optional=False)
    _check(load().gptq_pack_ordered(_ptr(codes), m, n, int(bits), _ptr(perm), _ptr(packed),
                                    _stream(stream)),
           "gptq_pack_ordered")


def gptq_dequant_gemm_workspace_size(tokens: int, m: int, n: int, has_perm: bool) -> int:
    out = _sz(0)
    _check(load().gptq_dequant_gemm_workspace_size(tokens, m, n, int(bool(has_perm)),
                                                   ctypes.byref(out)),
           "gptq_dequant_gemm_workspace_size")
    return out.value


def gptq_dequant_gemm(X, packed, bits: int, group_size: int, scales, zeros, Y, perm=None,
                      ws=None, stream=None) -> None:
    """Y[tokens, m] = X[tokens, n] W_q^T with W_q from processing-order packed codes."""
    tokens, n = X.shape
    m = packed.shape[0]
    d = X.device
    ng = _ngroups(n, group_size)
    _mat(packed, "packed", m, -(-(n * int(bits)) // 32), _INT32_LIKE, d)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _buf(perm, "perm", (n,), _INT32_LIKE, d)
    _mat(Y, "Y", tokens, m, ("float32", "bfloat16"), d)
    if ws is None:
        ws = _workspace(gptq_dequant_gemm_workspace_size(tokens, m, n, perm is not None),
                        X.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().gptq_dequant_gemm(_ptr(X), _dtype_code(X), tokens, n, _ld(X), _ptr(packed),
                                    _ld(packed), int(bits), int(group_size), _ptr(scales),
                                    _ptr(zeros), _ptr(perm), m, _ptr(Y), _dtype_code(Y), _ld(Y),
                                    _ptr(ws), nbytes, _stream(stream)),
           "gptq_dequant_gemm")


def gptq_dequantize(packed, bits: int, group_size: int, scales, zeros, n: int, W,
                    stream=None) -> None:
    """W[m, n] (bf16) = the product's weights from processing-order packed codes."""
    m = packed.shape[0]
    d = packed.device
    ng = _ngroups(int(n), group_size)
    _mat(packed, "packed", m, -(-(int(n) * int(bits)) // 32), _INT32_LIKE, d)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _mat(W, "W", m, int(n), ("bfloat16",), d)
    _check(load().gptq_dequantize(_ptr(packed), _ld(packed), int(bits), int(group_size),
                                  _ptr(scales), _ptr(zeros), m, int(n), _ptr(W), _ld(W),
                                  _stream(stream)),
           "gptq_dequantize")


def gptq_gemm_bf16(X, W, Y, stream=None) -> None:
    """Y[tokens, m] = X[tokens, n] W[m, n]^T (bf16 operands, Y fp32 or bf16)."""
    tokens, n = X.shape
    m = W.shape[0]
    _mat(W, "W", m, n, ("bfloat16",), X.device)
    _mat(Y, "Y", tokens, m, ("float32", "bfloat16"), X.device)
    _check(load().gptq_gemm_bf16(_ptr(X), tokens, n, _ld(X), _ptr(W), m, _ld(W), _ptr(Y),
                                 _dtype_code(Y), _ld(Y), _stream(stream)),
           "gptq_gemm_bf16")


def gptq_gather_columns(X, perm, Xp, stream=None) -> None:
    """Xp[t, p] = X[t, perm[p]] (bf16; Xp's columns past n are zeroed)."""
    tokens, n = X.shape
    _buf(perm, "perm", (n,), _INT32_LIKE, X.device, optional=False)
    _mat(Xp, "Xp", tokens, n, ("bfloat16",), X.device)
    _check(load().gptq_gather_columns(_ptr(X), _dtype_code(X), tokens, n, _ld(X), _ptr(perm),
                                      _ptr(Xp), _ld(Xp), _stream(stream)),
           "gptq_gather_columns")


def gptq_swiglu(gate, up, h, stream=None) -> None:
    """h[tokens, n] (bf16) = silu(gate) * up for fp32 gate, up."""
    tokens, n = gate.shape
    _mat(up, "up", tokens, n, ("float32",), gate.device)
    _mat(h, "h", tokens, n, ("bfloat16",), gate.device)
    _check(load().gptq_swiglu(_ptr(gate), _ld(gate), _ptr(up), _ld(up), tokens, n, _ptr(h),
                              _ld(h), _stream(stream)),
           "gptq_swiglu")


def gptq_residual_add(x, y, out, stream=None) -> None:
    """out[tokens, n] (bf16) = x (bf16) + y (fp32); out may be x."""
    tokens, n = x.shape
    _mat(y, "y", tokens, n, ("float32",), x.device)
    _mat(out, "out", tokens, n, ("bfloat16",), x.device)
    _check(load().gptq_residual_add(_ptr(x), _ld(x), _ptr(y), _ld(y), tokens, n, _ptr(out),
                                    _ld(out), _stream(stream)),
           "gptq_residual_add")


def awq_absum_workspace_size(n: int, tokens: int) -> int:
    out = _sz(0)
    _check(load().awq_absum_workspace_size(n, tokens, ctypes.byref(out)),
           "awq_absum_workspace_size")
    return out.value


def awq_lite_workspace_size(m: int, n: int) -> int:
    out = _sz(0)
    _check(load().awq_lite_workspace_size(m, n, ctypes.byref(out)), "awq_lite_workspace_size")
    return out.value


def awq_activation_absum(X, absum, ws=None, stream=None) -> None:
    """absum[n] += sum over tokens of |X[t, c]|."""
    tokens, n = X.shape
    _buf(absum, "absum", (n,), ("float32",), X.device, optional=False)
    if ws is None:
        ws = _workspace(awq_absum_workspace_size(n, tokens), X.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().awq_activation_absum(_ptr(X), _dtype_code(X), tokens, n, _ld(X), _ptr(absum),
                                       _ptr(ws), nbytes, _stream(stream)),
           "awq_activation_absum")


def awq_lite(W, S, absum, tokens: int, bits: int, group_size: int, s_out, alpha_out, losses,
             sym: bool = False, ws=None, stream=None) -> None:
    """alpha search; s_out[n], alpha_out[1], losses[n_alpha] fp32 device tensors."""
    m, n = W.shape
    d = W.device
    _mat(S, "S", n, n, ("float32",), d)
    _buf(absum, "absum", (n,), ("float32",), d, optional=False)
    _buf(s_out, "s_out", (n,), ("float32",), d, optional=False)
    _buf(alpha_out, "alpha_out", (1,), ("float32",), d, optional=False)
    _buf(losses, "losses", (1,), ("float32",), d, optional=False)
    if ws is None:
        ws = _workspace(awq_lite_workspace_size(m, n), W.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().awq_lite(_ptr(W), _dtype_code(W), m, n, _ld(W), _ptr(S), _ld(S), _ptr(absum),
                           int(tokens), int(bits), int(group_size), int(sym), losses.numel(),
                           _ptr(s_out), _ptr(alpha_out), _ptr(losses), _ptr(ws), nbytes,
                           _stream(stream)),
           "awq_lite")


def awq_clip_quantize(W, S, s, bits: int, group_size: int, codes, scales, zeros, clip_idx=None,
                      sym: bool = False, n_steps: int = 11, stream=None) -> None:
    m, n = W.shape
    d = W.device
    ng = _ngroups(n, group_size)
    _mat(S, "S", n, n, ("float32",), d)
    _buf(s, "s", (n,), ("float32",), d)
    _buf(codes, "codes", (m, n), ("uint8",), d, optional=False)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _buf(clip_idx, "clip_idx", (m, ng), ("uint8",), d)
    _check(load().awq_clip_quantize(_ptr(W), _dtype_code(W), m, n, _ld(W), _ptr(S), _ld(S),
                                    _ptr(s), int(bits), int(group_size), int(sym), int(n_steps),
                                    _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(clip_idx),
                                    _stream(stream)),
           "awq_clip_quantize")


def rtn_minmax(W, bits: int, group_size: int, codes, scales, zeros, sym: bool = False,
               stream=None) -> None:
    m, n = W.shape
    d = W.device
    ng = _ngroups(n, group_size)
    _buf(codes, "codes", (m, n), ("uint8",), d, optional=False)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _check(load().rtn_minmax(_ptr(W), _dtype_code(W), m, n, _ld(W), int(bits), int(group_size),
                             int(sym), _ptr(codes), _ptr(scales), _ptr(zeros), _stream(stream)),
           "rtn_minmax")


def gptq_layer_error_workspace_size(m: int, n: int) -> int:
    out = _sz()
    _check(load().gptq_layer_error_workspace_size(int(m), int(n), ctypes.byref(out)),
           "gptq_layer_error_workspace_size")
    return int(out.value)


def gptq_layer_error(W, codes, scales, zeros, g_idx, S, err, ws=None, stream=None) -> None:
    """err[m] (float64) = per-row output error delta_r S delta_r^T of the quantized layer."""
    m, n = W.shape
    d = W.device
    ng = scales.shape[1] if scales.dim() == 2 else 0
    _buf(codes, "codes", (m, n), ("uint8",), d, optional=False)
    _buf(scales, "scales", (m, ng), ("float32",), d, optional=False)
    _buf(zeros, "zeros", (m, ng), ("float32",), d, optional=False)
    _buf(g_idx, "g_idx", (n,), _INT32_LIKE, d, optional=False)
    _mat(S, "S", n, n, ("float32",), d)
    _buf(err, "err", (m,), ("float64",), d, optional=False)
    if ws is None:
        ws = _workspace(gptq_layer_error_workspace_size(m, n), d, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().gptq_layer_error(_ptr(W), _dtype_code(W), m, n, _ld(W), _ptr(codes),
                                   _ptr(scales), _ptr(zeros), int(ng), _ptr(g_idx), _ptr(S),
                                   _ld(S), _ptr(err), _ptr(ws), nbytes, _stream(stream)),
           "gptq_layer_error")


# ---------------------------------------------------------------------------
# 8-bit floating point, the quantized cache, log probabilities
# ---------------------------------------------------------------------------
# torch dtype -> one letter; filled on first use (this module does not import
# torch before it is needed)
_KIND = {}
_FLOAT = {"b": GPTQ_BF16, "f": GPTQ_F32}


def _on_gpu(t, name: str):
    """The device of an operand, which has to be a GPU."""
    if not _KIND:
        import torch

        _KIND.update({torch.bfloat16: "b", torch.float32: "f", torch.float8_e4m3fn: "8",
                      torch.uint8: "u", torch.int64: "l", torch.int32: "i"})
    d = t.device
    if d.type != "cuda":
        raise ValueError(f"{name} is on {d}, expected a GPU tensor")
    return d


def _plane(t, name: str, rows: int, cols: int, kinds: str, device, exact: str = "") -> int:
    """Checks a 2-D operand (unit column stride, at least rows x cols, on
    ``device``, a dtype among ``kinds``) and returns its row stride.  ``exact``: "r" and
    "c" for rows and columns that have to be as many as stated -- an operand's, where
    more of them mean that it belongs to another product; outputs may be larger."""
    if t is None:
        raise ValueError(f"{name} is required")
    if _KIND.get(t.dtype, "?") not in kinds:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] < cols or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: expected a 2-D tensor of at least {rows} x {cols} with unit "
                         f"column stride, got shape {tuple(shape)} strides {stride}")
    if exact and (("r" in exact and shape[0] != rows) or ("c" in exact and shape[1] != cols)):
        raise ValueError(f"{name}: expected {rows} x {cols}, got shape {tuple(shape)}")
    # the stride of a single row is not meaningful
    return stride[0] if shape[0] > 1 else max(stride[0], shape[1])


def _launch(name: str, device, stream, *args) -> None:
    """Calls an entry point on ``stream`` (default: the current stream of the
    tensors' device), with that device current."""
    import torch

    c = torch._C
    index = device.index
    if stream is None:
        raw = c._cuda_getCurrentRawStream(index)
    else:
        if stream.device != device:
            raise ValueError(f"{name}: the stream is on {stream.device}, the tensors on {device}")
        raw = stream.cuda_stream
    if index == c._cuda_getDevice():
        status = getattr(_lib, name)(*args, raw)
    else:
        with torch.cuda.device(index):
            status = getattr(_lib, name)(*args, raw)
    if status:
        _check(status, name)


@functools.lru_cache(maxsize=1024)
def _size_of(name: str, *args) -> int:
    """A workspace query by its arguments (what it answers depends on nothing else)."""
    out = _sz(0)
    _check(getattr(load(), name)(*args, ctypes.byref(out)), name)
    return out.value


def _space(need: int, ws, device, stream):
    """(pointer, bytes, tensor) of the caller's workspace, or of one for this call."""
    if ws is None:
        if not need:
            return None, 0, None
        ws = _workspace(need, device, stream)
        return ws.data_ptr(), need, ws
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def fp8_quantize_rows(X, codes, scales, stream=None) -> None:
    """codes[tokens, n] (e4m3 or uint8) and scales[ceil(n / 128), tokens] (fp32) of
    X[tokens, n] (bf16 or fp32): one scale per token and 128 columns."""
    tokens, n = X.shape
    d = _on_gpu(X, "X")
    ldx = _plane(X, "X", tokens, n, "bf", d)
    ldc = _plane(codes, "codes", tokens, n, "8u", d)
    lds = _plane(scales, "scales", -(-n // FP8_BLOCK), tokens, "f", d)
    _launch("fp8_quantize_rows", d, stream, X.data_ptr(), _FLOAT[_KIND[X.dtype]], tokens, n, ldx,
            codes.data_ptr(), ldc, scales.data_ptr(), lds)


def fp8_swiglu_quantize(gate, up, codes, scales, stream=None) -> None:
    """fp8_quantize_rows of silu(gate) * up (both bf16 or both fp32, [tokens, n])."""
    tokens, n = gate.shape
    d = _on_gpu(gate, "gate")
    ldg = _plane(gate, "gate", tokens, n, "bf", d)
    ldu = _plane(up, "up", tokens, n, _KIND[gate.dtype], d, "rc")
    ldc = _plane(codes, "codes", tokens, n, "8u", d)
    lds = _plane(scales, "scales", -(-n // FP8_BLOCK), tokens, "f", d)
    _launch("fp8_swiglu_quantize", d, stream, gate.data_ptr(), ldg, up.data_ptr(), ldu,
            _FLOAT[_KIND[gate.dtype]], tokens, n, codes.data_ptr(), ldc, scales.data_ptr(), lds)


def fp8_quantize_blocks(W, codes, scales, stream=None) -> None:
    """codes[m, n] (e4m3 or uint8) and scales[ceil(m / 128), ceil(n / 128)] (fp32) of
    W[m, n] (bf16 or fp32): one scale per 128 x 128 block."""
    m, n = W.shape
    d = _on_gpu(W, "W")
    ldw = _plane(W, "W", m, n, "bf", d)
    ldc = _plane(codes, "codes", m, n, "8u", d)
    lds = _plane(scales, "scales", -(-m // FP8_BLOCK), -(-n // FP8_BLOCK), "f", d)
    _launch("fp8_quantize_blocks", d, stream, W.data_ptr(), _FLOAT[_KIND[W.dtype]], m, n, ldw,
            codes.data_ptr(), ldc, scales.data_ptr(), lds)


def fp8_gemm_workspace_size(tokens: int, m: int, n: int) -> int:
    return _size_of("fp8_gemm_workspace_size", tokens, m, n)


def fp8_linear_workspace_size(tokens: int, m: int, n: int) -> int:
    return _size_of("fp8_linear_workspace_size", tokens, m, n)


def fp8_gemm(X, xscales, W, wscales, Y, residual=None, ws=None, stream=None) -> None:
    """Y[tokens, m] (fp32 or bf16) = X W^T of block-scaled e4m3 operands: X[tokens, n] with
    xscales[ceil(n / 128), tokens] (it may hold more tokens), W[m, n] with
    wscales[ceil(m / 128), ceil(n / 128)]; plus residual[tokens, m] (Y's type, may be Y) where
    it is given.  Y may have more rows and columns, which are left alone."""
    tokens, n = X.shape
    m = W.shape[0]
    d = _on_gpu(X, "X")
    nb = -(-n // FP8_BLOCK)
    ldx = _plane(X, "X", tokens, n, "8u", d)
    ldxs = _plane(xscales, "xscales", nb, tokens, "f", d, "r")
    ldw = _plane(W, "W", m, n, "8u", d, "rc")
    ldws = _plane(wscales, "wscales", -(-m // FP8_BLOCK), nb, "f", d, "rc")
    ldy = _plane(Y, "Y", tokens, m, "bf", d)
    ldr = 0
    if residual is not None:
        ldr = _plane(residual, "residual", tokens, m, _KIND[Y.dtype], d,
                     "" if residual.shape == Y.shape else "rc")
    p, nbytes, ws = _space(fp8_gemm_workspace_size(tokens, m, n), ws, d, stream)
    _launch("fp8_gemm", d, stream, X.data_ptr(), tokens, n, ldx, xscales.data_ptr(), ldxs,
            W.data_ptr(), m, ldw, wscales.data_ptr(), ldws, _ptr(residual), ldr, Y.data_ptr(),
            _FLOAT[_KIND[Y.dtype]], ldy, p, nbytes)


def fp8_linear(X, W, wscales, Y, ws=None, stream=None) -> None:
    """Y[tokens, m] (fp32 or bf16) = X W^T with X[tokens, n] (bf16 or fp32) quantized as by
    fp8_quantize_rows and W[m, n] e4m3 with wscales[ceil(m / 128), ceil(n / 128)]."""
    tokens, n = X.shape
    m = W.shape[0]
    d = _on_gpu(X, "X")
    ldx = _plane(X, "X", tokens, n, "bf", d)
    ldw = _plane(W, "W", m, n, "8u", d, "rc")
    ldws = _plane(wscales, "wscales", -(-m // FP8_BLOCK), -(-n // FP8_BLOCK), "f", d, "rc")
    ldy = _plane(Y, "Y", tokens, m, "bf", d)
    p, nbytes, ws = _space(fp8_linear_workspace_size(tokens, m, n), ws, d, stream)
    _launch("fp8_linear", d, stream, X.data_ptr(), _FLOAT[_KIND[X.dtype]], tokens, n, ldx,
            W.data_ptr(), m, ldw, wscales.data_ptr(), ldws, Y.data_ptr(), _FLOAT[_KIND[Y.dtype]], ldy, p, nbytes)


def fp8_gated_gemm_workspace_size(tokens: int, m: int, n: int) -> int:
    return _size_of("fp8_gated_gemm_workspace_size", tokens, m, n)


def fp8_gated_gemm(X, xscales, Wg, gscales, Wu, uscales, codes, scales, ws=None,
                   stream=None) -> None:
    """codes[tokens, m] and scales[ceil(m / 128), tokens] of silu(X Wg^T) * (X Wu^T), the
    products (operands as in fp8_gemm) rounded to bf16; codes apart from X."""
    tokens, n = X.shape
    m = Wg.shape[0]
    d = _on_gpu(X, "X")
    nb, mb = -(-n // FP8_BLOCK), -(-m // FP8_BLOCK)
    ldx = _plane(X, "X", tokens, n, "8u", d)
    ldxs = _plane(xscales, "xscales", nb, tokens, "f", d, "r")
    ldwg = _plane(Wg, "Wg", m, n, "8u", d, "rc")
    ldgs = _plane(gscales, "gscales", mb, nb, "f", d, "rc")
    ldwu = _plane(Wu, "Wu", m, n, "8u", d, "rc")
    ldus = _plane(uscales, "uscales", mb, nb, "f", d, "rc")
    ldc = _plane(codes, "codes", tokens, m, "8u", d)
    lds = _plane(scales, "scales", mb, tokens, "f", d)
    p, nbytes, ws = _space(fp8_gated_gemm_workspace_size(tokens, m, n), ws, d, stream)
    _launch("fp8_gated_gemm", d, stream, X.data_ptr(), tokens, n, ldx, xscales.data_ptr(), ldxs,
            Wg.data_ptr(), m, ldwg, gscales.data_ptr(), ldgs, Wu.data_ptr(), ldwu,
            uscales.data_ptr(), ldus, codes.data_ptr(), ldc, scales.data_ptr(), lds, p, nbytes)


def make_kv_cache(codes, scales, zeros, head_dim: int, fmt: str = "int8",
                  group_size: int = 128) -> GPTQKVCache:
    """The handle of a paged cache of keys or of values.

    codes: uint8 [pages, page_size, heads, bytes], bytes = head_dim (int8, e4m3) or
    head_dim / 2 (int4); scales: fp32 [pages, page_size, heads, groups]; zeros: uint8 of the
    scales' shape and strides (integers with zero-points), or None.  Pages, slots and heads
    may lie in any order; the last dimension is dense."""
    if fmt not in _KV_FORMATS:
        raise ValueError(f"fmt: {fmt!r}, expected one of {tuple(_KV_FORMATS)}")
    head_dim, group_size = int(head_dim), int(group_size)
    d = _on_gpu(codes, "codes")
    nbytes = head_dim // 2 if fmt == "int4" else head_dim
    groups = 1 if group_size <= 0 else -(-head_dim // group_size)
    if _KIND.get(codes.dtype) not in ("u", "8"):
        raise TypeError(f"codes: unsupported dtype {codes.dtype}")
    if _KIND.get(scales.dtype) != "f":
        raise TypeError(f"scales: dtype {scales.dtype}, expected float32")
    shape, cs, ps = codes.shape, codes.stride(), scales.stride()
    if len(shape) != 4 or shape[3] != nbytes or cs[3] != 1:
        raise ValueError(f"codes: shape {tuple(shape)} strides {cs}, expected "
                         f"[pages, page_size, heads, {nbytes}] with a dense last dimension")
    pages, page_size, heads = shape[:3]
    want = (pages, page_size, heads, groups)
    if scales.device != d:
        raise ValueError(f"scales is on {scales.device}, expected {d}")
    if scales.shape != want or (ps[3] != 1 and groups > 1):
        raise ValueError(f"scales: shape {tuple(scales.shape)} strides {ps}, expected {want} with "
                         "a dense last dimension")
    z = None
    if zeros is not None:
        if fmt == "e4m3":
            raise ValueError("zeros: e4m3 has none")
        if _KIND.get(zeros.dtype) != "u":
            raise TypeError(f"zeros: dtype {zeros.dtype}, expected uint8")
        if zeros.device != d:
            raise ValueError(f"zeros is on {zeros.device}, expected {d}")
        if zeros.shape != want or zeros.stride() != ps:
            raise ValueError("zeros must have the shape and strides of scales")
        z = zeros.data_ptr()
    c = GPTQKVCache(codes.data_ptr(), scales.data_ptr(), z, pages, cs[0], cs[1], cs[2], ps[0],
                    ps[1], ps[2], page_size, heads, head_dim, group_size, _KV_FORMATS[fmt])
    c.tensors = (codes, scales, zeros)
    c.device = d
    c.row = (heads, head_dim)
    c.paging = (pages, page_size)
    c.ref = ctypes.addressof(c)
    return c


_KV_NONE = (None, 0, 0)


def _kv_rows(t, name: str, cache: Optional[GPTQKVCache], tokens: int, device, dtype):
    """(pointer, token stride, head stride) of rows [tokens, heads, head_dim]."""
    if cache is None or t is None:
        if cache is None and t is None:
            return _KV_NONE
        raise ValueError(f"{name}: rows and their cache come together")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype} for keys and values alike")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or stride[2] != 1 or shape[0] != tokens or shape[1:] != cache.row:
        raise ValueError(f"{name}: shape {tuple(shape)} strides {stride}, expected "
                         f"{(tokens, *cache.row)} with a dense last dimension")
    if cache.device != device or t.device != device:
        raise ValueError(f"{name}: rows on {t.device}, cache on {cache.device}, "
                         f"expected {device}")
    return t.data_ptr(), stride[0], stride[1]


def _kv_call(K, V, slots, kc, vc, info):
    rows = K if K is not None else V
    if rows is None:
        raise ValueError("keys with their cache or values with theirs are required")
    d = _on_gpu(slots, "slots")
    if _KIND.get(slots.dtype) != "l" or slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots: expected a contiguous 1-D int64 tensor")
    if info is not None:
        _buf(info, "info", (1,), ("int32",), d)
    dtype = rows.dtype
    dt = _FLOAT.get(_KIND.get(dtype))
    if dt is None:
        raise TypeError(f"rows: dtype {dtype}, expected bfloat16 or float32")
    tokens = slots.shape[0]
    k = _kv_rows(K, "K", kc, tokens, d, dtype)
    v = _kv_rows(V, "V", vc, tokens, d, dtype)
    if kc is not None and vc is not None and kc.paging != vc.paging:
        raise ValueError("the two caches differ in pages or page_size")
    return d, tokens, k, v, dt, None if kc is None else kc.ref, None if vc is None else vc.ref


def kv_cache_write_workspace_size(tokens: int, cache: GPTQKVCache) -> int:
    out = _sz(0)
    _check(load().kv_cache_write_workspace_size(tokens, ctypes.byref(cache), ctypes.byref(out)),
           "kv_cache_write_workspace_size")
    return out.value


def kv_cache_write(K, V, slots, kc, vc, info=None, ws=None, stream=None) -> None:
    """Quantize rows K, V [tokens, heads, head_dim] (bf16 or fp32) into slots[tokens] (int64,
    negative: padding, not written) of the caches kc, vc (either may be None with its rows)."""
    d, tokens, (kp, kt, kh), (vp, vt, vh), dt, pk, pv = _kv_call(K, V, slots, kc, vc, info)
    need = 0
    if ws is None and tokens > GPTQ_KV_SMALL_TOKENS:
        need = kv_cache_write_workspace_size(tokens, kc if kc is not None else vc)
    p, nbytes, ws = _space(need, ws, d, stream)
    _launch("kv_cache_write", d, stream, kp, kt, kh, vp, vt, vh, dt, tokens, slots.data_ptr(), pk,
            pv, _ptr(info), p, nbytes)


def kv_cache_read(kc, vc, slots, K, V, info=None, stream=None) -> None:
    """Rows K, V [tokens, heads, head_dim] (bf16 or fp32) = the caches' values at slots[tokens]
    (int64, negative: zeros)."""
    d, tokens, (kp, kt, kh), (vp, vt, vh), dt, pk, pv = _kv_call(K, V, slots, kc, vc, info)
    _launch("kv_cache_read", d, stream, pk, pv, slots.data_ptr(), tokens, kp, kt, kh, vp, vt, vh,
            dt, _ptr(info))


def token_logprobs_workspace_size(tokens: int, vocab: int, top: int) -> int:
    return _size_of("token_logprobs_workspace_size", tokens, vocab, top)


def _vector(t, name: str, count: int, kind: str, device, optional: bool = True) -> None:
    """A contiguous buffer of at least ``count`` elements."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if _KIND.get(t.dtype) != kind:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous() or t.numel() < count:
        raise ValueError(f"{name}: expected {count} contiguous elements, got shape "
                         f"{tuple(t.shape)} strides {t.stride()}")


def token_logprobs(logits, ids, logprob, entropy=None, top_ids=None, top_logprobs=None, ws=None,
                   stream=None) -> None:
    """For each row of logits[tokens, vocab] (bf16 or fp32): logprob[tokens] of ids[tokens]
    (int64, negative: not asked for, 0; either both or neither given), entropy[tokens], and the
    top alternatives top_ids (int32) and top_logprobs [tokens, top], top <= 32."""
    tokens, vocab = logits.shape
    d = _on_gpu(logits, "logits")
    ldl = _plane(logits, "logits", tokens, vocab, "bf", d)
    _vector(ids, "ids", tokens, "l", d, optional=logprob is None)
    _vector(logprob, "logprob", tokens, "f", d, optional=ids is None)
    _vector(entropy, "entropy", tokens, "f", d)
    top = 0
    if top_ids is not None or top_logprobs is not None:
        if top_ids is None or top_ids.dim() != 2:
            raise ValueError("top_ids: expected [tokens, top] together with top_logprobs")
        top = top_ids.shape[1]
        if top_logprobs is None or top_logprobs.shape != top_ids.shape:
            raise ValueError("top_logprobs: expected the shape of top_ids")
        _vector(top_ids, "top_ids", tokens * top, "i", d)
        _vector(top_logprobs, "top_logprobs", tokens * top, "f", d)
    p, nbytes, ws = _space(token_logprobs_workspace_size(tokens, vocab, top), ws, d, stream)
    _launch("token_logprobs", d, stream, logits.data_ptr(), _FLOAT[_KIND[logits.dtype]], tokens,
            vocab, ldl, _ptr(ids), _ptr(logprob), _ptr(entropy), top, _ptr(top_ids), _ptr(top_logprobs),
            p, nbytes)
