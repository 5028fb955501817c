"""ctypes binding of libpackedbitgemv.so.

Argument marshalling only: every function checks tensor placement, dtype and
shape, passes raw device pointers and the current HIP stream to the C entry
point of the same name, and raises PbgError on a nonzero return code. All
computation happens in the library's HIP kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

import torch

from .build import LIB_PATH

PBG_ERR_CODE = -4
ARGMAX_KEYS_PER_ROW = 4096  # PBG_ARGMAX_KEYS_PER_ROW
MAX_M = 8  # PBG_MAX_M
STREAM_READ_SINK_WORDS = 8192  # PBG_STREAM_READ_SINK_WORDS
LOGITS_SLICE = 1024  # PBG_LOGITS_SLICE

_c_int = ctypes.c_int
_c_i64 = ctypes.c_int64
_vp = ctypes.c_void_p

# (restype, argtypes) of every entry point declared in include/packed_bit_gemv.h.
_SIGNATURES = {
    "pbg_abi_version": (_c_int, []),
    "pbg_strerror": (ctypes.c_char_p, [_c_int]),
    "pbg_words_per_row": (_c_i64, [_c_i64]),
    "pack_ternary": (_c_int, [_vp, _c_i64, _c_i64, _vp, _vp, _vp, _vp, _vp]),
    "ternary_gemv": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "ternary_gemm_small": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp]),
    "pbg_words_per_row3": (_c_i64, [_c_i64]),
    "pack_ternary3": (_c_int, [_vp, _c_i64, _c_i64, _vp, _vp, _vp, _vp, _vp]),
    "ternary3_gemv": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "ternary3_gemm_small": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp]),
    "pbg_splitk_workspace_bytes": (_c_i64, [_c_i64, _c_i64]),
    "ternary_gemm_splitk": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _c_i64, _vp]),
    "int8_head_gemv": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp]),
    "int8_head_argmax": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _vp, _vp]),
    "int8_head_argmax_noalloc": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _vp]),
    "int8_embedding_gather": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp]),
    "ternary_swiglu_gate_up": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "ternary_ffn_swiglu": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _vp, _vp]),
    "ternary_swiglu_gate_up_small": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp]),
    "ternary_ffn_swiglu_small": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp,
                                          _vp]),
    "ternary3_ffn_swiglu_small": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp,
                                           _vp]),
    "ternary3_swiglu_gate_up": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "ternary3_ffn_swiglu": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _vp, _vp]),
    "ternary3_swiglu_gate_up_small": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp]),
    "pbg_q8_row_bytes": (_c_i64, [_c_i64]),
    "add_rmsnorm": (_c_int, [_vp, _vp, _vp, ctypes.c_float, _c_i64, _c_i64, _vp, _vp, _vp, _vp, _vp]),
    "quantize_rows": (_c_int, [_vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "ternary_gemm_i8": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _vp, _c_i64, _vp, _vp]),
    "ternary_swiglu_gate_up_i8": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _c_i64, _vp, _vp]),
    "pbg_lora_workspace_bytes": (_c_i64, [_c_i64, _c_i64]),
    "lora_add": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _vp, _c_i64,
                          _vp]),
    "cache_plan": (_c_int, [_vp, _vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _vp,
                            _vp, _vp, _vp, _vp]),
    "rotary_qkv": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float, _c_int, _c_i64, _c_i64, _c_i64,
                            _c_i64, _c_i64, _vp, _vp, _vp, _c_i64, _c_i64, _vp]),
    "pbg_attention_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64]),
    "tree_attention": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _c_i64, _vp, _c_i64, _c_i64,
                                _c_i64, _c_i64, ctypes.c_float, _vp, _vp, _c_i64, _vp]),
    "penalize_logits": (_c_int, [_vp, _vp, _vp, _c_i64, _vp, _vp, _vp, _vp, _vp, _c_i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _c_i64, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp, _vp, _vp, _vp, _c_i64, _vp]),
    "pbg_stream_read": (_c_int, [_vp, _c_i64, _vp, _vp]),
}


class PbgError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {msg} ({code})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m packed_bit_gemv_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/packed_bit_gemv.h."""
    path = os.path.join(os.path.dirname(os.path.dirname(LIB_PATH)), "include", "packed_bit_gemv.h")
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\**\s*([A-Za-z_][A-Za-z0-9_]*)\s*\(", text, flags=re.M)


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise PbgError(fn, rc, lib().pbg_strerror(rc).decode())


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def words_per_row(k: int) -> int:
    return int(lib().pbg_words_per_row(int(k)))


def pack_ternary(codes: torch.Tensor, packed: torch.Tensor | None = None, row_sum: torch.Tensor | None = None,
                 stats: torch.Tensor | None = None, check: bool = True):
    """Pack int8 codes [n, k] on the GPU. Returns (packed, row_sum, stats).

    stats holds n_minus, n_zero, n_plus, n_invalid. With check=True the call
    waits for the stream and raises PbgError if any code is outside {-1,0,1}.
    """
    _dev(codes, "codes", torch.int8)
    if codes.dim() != 2:
        raise ValueError("codes must be [n, k]")
    n, k = codes.shape
    dev = codes.device
    if packed is None:
        packed = torch.empty((n, words_per_row(k)), dtype=torch.int32, device=dev)
    if row_sum is None:
        row_sum = torch.empty((n,), dtype=torch.int32, device=dev)
    if stats is None:
        stats = torch.empty((4,), dtype=torch.int64, device=dev)
    _dev(packed, "packed", torch.int32)
    _dev(row_sum, "row_sum", torch.int32)
    _dev(stats, "stats", torch.int64)
    if tuple(packed.shape) != (n, words_per_row(k)) or tuple(row_sum.shape) != (n,) or stats.numel() != 4:
        raise ValueError("output shapes do not match codes")
    host = (ctypes.c_int64 * 4)() if check else None
    rc = lib().pack_ternary(codes.data_ptr(), n, k, packed.data_ptr(), row_sum.data_ptr(), stats.data_ptr(),
                            ctypes.addressof(host) if host is not None else None, _stream(codes))
    _check("pack_ternary", rc)
    return packed, row_sum, stats


def _ternary_args(packed, scale, k, x):
    _dev(packed, "packed", torch.int32)
    _dev(scale, "scale", torch.float32)
    _dev(x, "x", torch.float16)
    n = packed.shape[0]
    if packed.dim() != 2 or packed.shape[1] != words_per_row(k):
        raise ValueError(f"packed must be [n, {words_per_row(k)}] for k={k}")
    if tuple(scale.shape) != (n,):
        raise ValueError("scale must be [n]")
    return n


def ternary_gemv(packed: torch.Tensor, scale: torch.Tensor, k: int, x: torch.Tensor,
                 y: torch.Tensor | None = None) -> torch.Tensor:
    """y[r] = scale[r] * sum_j c[r, j] * x[j]; x is fp16 [k], y fp32 [n]."""
    n = _ternary_args(packed, scale, k, x)
    if tuple(x.shape) != (k,):
        raise ValueError(f"x must be [{k}]")
    if y is None:
        y = torch.empty((n,), dtype=torch.float32, device=packed.device)
    _dev(y, "y", torch.float32)
    if tuple(y.shape) != (n,):
        raise ValueError("y must be [n]")
    rc = lib().ternary_gemv(packed.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), y.data_ptr(), _stream(packed))
    _check("ternary_gemv", rc)
    return y


def ternary_gemm_small(packed: torch.Tensor, scale: torch.Tensor, k: int, x: torch.Tensor,
                       y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[i, r] = scale[r] * sum_j c[r, j] * X[i, j]; X fp16 [m, k], m <= 8; Y fp32 [m, n]."""
    n = _ternary_args(packed, scale, k, x)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [m, {k}]")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=packed.device)
    _dev(y, "y", torch.float32)
    if tuple(y.shape) != (m, n):
        raise ValueError("y must be [m, n]")
    rc = lib().ternary_gemm_small(packed.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), m, y.data_ptr(),
                                  _stream(packed))
    _check("ternary_gemm_small", rc)
    return y


def words_per_row3(k: int) -> int:
    return int(lib().pbg_words_per_row3(int(k)))


def pack_ternary3(codes: torch.Tensor, packed: torch.Tensor | None = None, row_sum: torch.Tensor | None = None,
                  stats: torch.Tensor | None = None, check: bool = True):
    """Pack five-level int8 codes [n, k] (-2..+2) on the GPU. Returns (packed, row_sum, stats).

    stats holds the counts of -2, -1, 0, +1, +2 and of invalid codes. With check=True the call
    waits for the stream and raises PbgError if any code is outside -2..+2.
    """
    _dev(codes, "codes", torch.int8)
    if codes.dim() != 2:
        raise ValueError("codes must be [n, k]")
    n, k = codes.shape
    dev = codes.device
    if packed is None:
        packed = torch.empty((n, words_per_row3(k)), dtype=torch.int32, device=dev)
    if row_sum is None:
        row_sum = torch.empty((n,), dtype=torch.int32, device=dev)
    if stats is None:
        stats = torch.empty((6,), dtype=torch.int64, device=dev)
    _dev(packed, "packed", torch.int32)
    _dev(row_sum, "row_sum", torch.int32)
    _dev(stats, "stats", torch.int64)
    if tuple(packed.shape) != (n, words_per_row3(k)) or tuple(row_sum.shape) != (n,) or stats.numel() != 6:
        raise ValueError("output shapes do not match codes")
    host = (ctypes.c_int64 * 6)() if check else None
    rc = lib().pack_ternary3(codes.data_ptr(), n, k, packed.data_ptr(), row_sum.data_ptr(), stats.data_ptr(),
                             ctypes.addressof(host) if host is not None else None, _stream(codes))
    _check("pack_ternary3", rc)
    return packed, row_sum, stats


def _ternary3_args(packed, scale, k, x):
    _dev(packed, "packed", torch.int32)
    _dev(scale, "scale", torch.float32)
    _dev(x, "x", torch.float16)
    n = packed.shape[0]
    if packed.dim() != 2 or packed.shape[1] != words_per_row3(k):
        raise ValueError(f"packed must be [n, {words_per_row3(k)}] for k={k}")
    if tuple(scale.shape) != (n,):
        raise ValueError("scale must be [n]")
    return n


def ternary3_gemv(packed: torch.Tensor, scale: torch.Tensor, k: int, x: torch.Tensor,
                  y: torch.Tensor | None = None) -> torch.Tensor:
    """Five-level y[r] = scale[r] * sum_j c[r, j] * x[j]; x fp16 [k], y fp32 [n]."""
    n = _ternary3_args(packed, scale, k, x)
    if tuple(x.shape) != (k,):
        raise ValueError(f"x must be [{k}]")
    if y is None:
        y = torch.empty((n,), dtype=torch.float32, device=packed.device)
    _dev(y, "y", torch.float32)
    if tuple(y.shape) != (n,):
        raise ValueError("y must be [n]")
    rc = lib().ternary3_gemv(packed.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), y.data_ptr(), _stream(packed))
    _check("ternary3_gemv", rc)
    return y


def ternary3_gemm_small(packed: torch.Tensor, scale: torch.Tensor, k: int, x: torch.Tensor,
                        y: torch.Tensor | None = None) -> torch.Tensor:
    """Five-level Y[i, r] = scale[r] * sum_j c[r, j] * X[i, j]; X fp16 [m, k], m <= 8; Y fp32 [m, n]."""
    n = _ternary3_args(packed, scale, k, x)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [m, {k}]")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=packed.device)
    _dev(y, "y", torch.float32)
    if tuple(y.shape) != (m, n):
        raise ValueError("y must be [m, n]")
    rc = lib().ternary3_gemm_small(packed.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), m, y.data_ptr(),
                                   _stream(packed))
    _check("ternary3_gemm_small", rc)
    return y


def splitk_workspace(n: int, k: int, device) -> torch.Tensor:
    """A zeroed workspace for ternary_gemm_splitk on [n, k] matrices (any m)."""
    nbytes = int(lib().pbg_splitk_workspace_bytes(int(n), int(k)))
    return torch.zeros(((nbytes + 7) // 8,), dtype=torch.int64, device=device)


def ternary_gemm_splitk(packed: torch.Tensor, scale: torch.Tensor, k: int, x: torch.Tensor, workspace: torch.Tensor,
                        y: torch.Tensor | None = None) -> torch.Tensor:
    """ternary_gemv (x [k] -> y [n]) or ternary_gemm_small (x [m, k] -> y [m, n]) with K split
    across workgroups; workspace from splitk_workspace(n, k), reused across calls."""
    n = _ternary_args(packed, scale, k, x)
    if x.dim() == 1 and x.shape[0] == k:
        m, y_shape = 1, (n,)
    elif x.dim() == 2 and x.shape[1] == k:
        m, y_shape = x.shape[0], (x.shape[0], n)
    else:
        raise ValueError(f"x must be [{k}] or [m, {k}]")
    if y is None:
        y = torch.empty(y_shape, dtype=torch.float32, device=packed.device)
    _dev(y, "y", torch.float32)
    if tuple(y.shape) != y_shape:
        raise ValueError(f"y must be {list(y_shape)}")
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA (HIP) tensor")
    rc = lib().ternary_gemm_splitk(packed.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), m, y.data_ptr(),
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream(packed))
    _check("ternary_gemm_splitk", rc)
    return y


def int8_head_gemv(w: torch.Tensor, scale: torch.Tensor, x: torch.Tensor,
                   y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[i, v] = scale[v] * sum_j w[v, j] * X[i, j]; w int8 [n, k], X fp16 [m, k]; Y fp32 [m, n]."""
    _dev(w, "w", torch.int8)
    _dev(scale, "scale", torch.float32)
    _dev(x, "x", torch.float16)
    if w.dim() != 2:
        raise ValueError("w must be [n, k]")
    n, k = w.shape
    if tuple(scale.shape) != (n,):
        raise ValueError("scale must be [n]")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [m, {k}]")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=w.device)
    _dev(y, "y", torch.float32)
    if tuple(y.shape) != (m, n):
        raise ValueError("y must be [m, n]")
    rc = lib().int8_head_gemv(w.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), m, y.data_ptr(), _stream(w))
    _check("int8_head_gemv", rc)
    return y


def int8_head_argmax(w: torch.Tensor, scale: torch.Tensor, x: torch.Tensor, keys: torch.Tensor | None = None,
                     token: torch.Tensor | None = None, logit: torch.Tensor | None = None):
    """Greedy token per activation row: (token int32 [m], logit fp32 [m]).

    keys is an int64 workspace of at least m * ARGMAX_KEYS_PER_ROW entries, zero before its first
    use and left zero by every call (a zeroed one is allocated if not given).
    """
    _dev(w, "w", torch.int8)
    _dev(scale, "scale", torch.float32)
    _dev(x, "x", torch.float16)
    if w.dim() != 2 or x.dim() != 2 or x.shape[1] != w.shape[1] or tuple(scale.shape) != (w.shape[0],):
        raise ValueError("w [n, k], scale [n], x [m, k]")
    n, k = w.shape
    m = x.shape[0]
    dev = w.device
    if keys is None:
        keys = torch.zeros((m * ARGMAX_KEYS_PER_ROW,), dtype=torch.int64, device=dev)
    if token is None:
        token = torch.empty((m,), dtype=torch.int32, device=dev)
    if logit is None:
        logit = torch.empty((m,), dtype=torch.float32, device=dev)
    _dev(keys, "keys", torch.int64)
    _dev(token, "token", torch.int32)
    _dev(logit, "logit", torch.float32)
    if keys.numel() < m * ARGMAX_KEYS_PER_ROW or token.numel() != m or logit.numel() != m:
        raise ValueError("keys holds m * ARGMAX_KEYS_PER_ROW entries, token and logit m")
    rc = lib().int8_head_argmax(w.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), m, keys.data_ptr(),
                                token.data_ptr(), logit.data_ptr(), _stream(w))
    _check("int8_head_argmax", rc)
    return token, logit


def int8_head_argmax_noalloc(w: torch.Tensor, scale: torch.Tensor, x: torch.Tensor,
                             token: torch.Tensor | None = None, logit: torch.Tensor | None = None):
    """int8_head_argmax with the library's own workspace: (token int32 [m], logit fp32 [m]).

    The C call allocates nothing (pass token and logit to keep this wrapper from allocating
    them). Calls that overlap in time on one GPU race.
    """
    _dev(w, "w", torch.int8)
    _dev(scale, "scale", torch.float32)
    _dev(x, "x", torch.float16)
    if w.dim() != 2 or x.dim() != 2 or x.shape[1] != w.shape[1] or tuple(scale.shape) != (w.shape[0],):
        raise ValueError("w [n, k], scale [n], x [m, k]")
    n, k = w.shape
    m = x.shape[0]
    if token is None:
        token = torch.empty((m,), dtype=torch.int32, device=w.device)
    if logit is None:
        logit = torch.empty((m,), dtype=torch.float32, device=w.device)
    _dev(token, "token", torch.int32)
    _dev(logit, "logit", torch.float32)
    if token.numel() != m or logit.numel() != m:
        raise ValueError("token and logit hold m entries")
    rc = lib().int8_head_argmax_noalloc(w.data_ptr(), scale.data_ptr(), n, k, x.data_ptr(), m, token.data_ptr(),
                                        logit.data_ptr(), _stream(w))
    _check("int8_head_argmax_noalloc", rc)
    return token, logit


def int8_embedding_gather(table: torch.Tensor, scale: torch.Tensor, tokens: torch.Tensor,
                          out: torch.Tensor | None = None) -> torch.Tensor:
    """Rows scale[t] * table[t] (fp32 [m, k]) for int32 token ids; ids outside [0, n) give NaN rows."""
    _dev(table, "table", torch.int8)
    _dev(scale, "scale", torch.float32)
    _dev(tokens, "tokens", torch.int32)
    if table.dim() != 2 or tokens.dim() != 1 or tuple(scale.shape) != (table.shape[0],):
        raise ValueError("table [n, k], scale [n], tokens [m]")
    n, k = table.shape
    m = tokens.shape[0]
    if out is None:
        out = torch.empty((m, k), dtype=torch.float32, device=table.device)
    _dev(out, "out", torch.float32)
    if tuple(out.shape) != (m, k):
        raise ValueError("out must be [m, k]")
    rc = lib().int8_embedding_gather(table.data_ptr(), scale.data_ptr(), n, k, tokens.data_ptr(), m,
                                     out.data_ptr(), _stream(table))
    _check("int8_embedding_gather", rc)
    return out


def _ffn_rows(x: torch.Tensor, d_model: int) -> int:
    """0 for x [d_model] (one row), m for x [m, d_model] with 1 <= m <= 8."""
    if x.dim() == 1 and tuple(x.shape) == (d_model,):
        return 0
    if x.dim() == 2 and x.shape[1] == d_model and 1 <= x.shape[0] <= MAX_M:
        return x.shape[0]
    raise ValueError(f"x must be [{d_model}] or [m, {d_model}] with 1 <= m <= {MAX_M}")


def _swiglu_gate_up(prefix: str, wpr, gate, gate_scale, up, up_scale, d_model, x, h):
    for t, name in ((gate, "gate"), (up, "up")):
        _dev(t, name, torch.int32)
    for t, name in ((gate_scale, "gate_scale"), (up_scale, "up_scale")):
        _dev(t, name, torch.float32)
    _dev(x, "x", torch.float16)
    d_ff = gate.shape[0]
    if gate.dim() != 2 or tuple(up.shape) != tuple(gate.shape) or gate.shape[1] != wpr(d_model):
        raise ValueError(f"gate and up must be [d_ff, {wpr(d_model)}]")
    if tuple(gate_scale.shape) != (d_ff,) or tuple(up_scale.shape) != (d_ff,):
        raise ValueError("scales must be [d_ff]")
    m = _ffn_rows(x, d_model)
    h_shape = (d_ff,) if m == 0 else (m, d_ff)
    if h is None:
        h = torch.empty(h_shape, dtype=torch.float16, device=gate.device)
    _dev(h, "h", torch.float16)
    if tuple(h.shape) != h_shape:
        raise ValueError(f"h must be {list(h_shape)}")
    if m == 0:
        name = f"{prefix}_swiglu_gate_up"
        rc = getattr(lib(), name)(gate.data_ptr(), gate_scale.data_ptr(), up.data_ptr(), up_scale.data_ptr(),
                                  d_model, d_ff, x.data_ptr(), h.data_ptr(), _stream(gate))
    else:
        name = f"{prefix}_swiglu_gate_up_small"
        rc = getattr(lib(), name)(gate.data_ptr(), gate_scale.data_ptr(), up.data_ptr(), up_scale.data_ptr(),
                                  d_model, d_ff, x.data_ptr(), m, h.data_ptr(), _stream(gate))
    _check(name, rc)
    return h


def ternary_swiglu_gate_up(gate: torch.Tensor, gate_scale: torch.Tensor, up: torch.Tensor, up_scale: torch.Tensor,
                           d_model: int, x: torch.Tensor, h: torch.Tensor | None = None) -> torch.Tensor:
    """h = fp16(silu(gate x) * up x) in one launch; gate, up packed [d_ff, words_per_row(d_model)].

    x fp16 [d_model] gives h [d_ff]; x [m, d_model] (m <= 8, one weight read for all rows) gives h [m, d_ff].
    """
    return _swiglu_gate_up("ternary", words_per_row, gate, gate_scale, up, up_scale, d_model, x, h)


def ternary3_swiglu_gate_up(gate: torch.Tensor, gate_scale: torch.Tensor, up: torch.Tensor, up_scale: torch.Tensor,
                            d_model: int, x: torch.Tensor, h: torch.Tensor | None = None) -> torch.Tensor:
    """ternary_swiglu_gate_up with gate and up in the 3-bit layout, packed [d_ff, words_per_row3(d_model)]."""
    return _swiglu_gate_up("ternary3", words_per_row3, gate, gate_scale, up, up_scale, d_model, x, h)


def _ffn_swiglu(prefix: str, wpr, gate, gate_scale, up, up_scale, down, down_scale, x, h, y):
    for t, name in ((gate, "gate"), (up, "up"), (down, "down")):
        _dev(t, name, torch.int32)
    for t, name in ((gate_scale, "gate_scale"), (up_scale, "up_scale"), (down_scale, "down_scale")):
        _dev(t, name, torch.float32)
    _dev(x, "x", torch.float16)
    d_ff, d_model = gate.shape[0], down.shape[0]
    if gate.dim() != 2 or tuple(up.shape) != tuple(gate.shape) or gate.shape[1] != wpr(d_model):
        raise ValueError(f"gate and up must be [d_ff, {wpr(d_model)}]")
    if down.dim() != 2 or down.shape[1] != wpr(d_ff):
        raise ValueError(f"down must be [d_model, {wpr(d_ff)}]")
    if tuple(gate_scale.shape) != (d_ff,) or tuple(up_scale.shape) != (d_ff,) or tuple(down_scale.shape) != (d_model,):
        raise ValueError("scales must be [d_ff], [d_ff], [d_model]")
    m = _ffn_rows(x, d_model)
    h_shape = (d_ff,) if m == 0 else (m, d_ff)
    y_shape = (d_model,) if m == 0 else (m, d_model)
    dev = gate.device
    if h is None:
        h = torch.empty(h_shape, dtype=torch.float16, device=dev)
    if y is None:
        y = torch.empty(y_shape, dtype=torch.float32, device=dev)
    _dev(h, "h", torch.float16)
    _dev(y, "y", torch.float32)
    if tuple(h.shape) != h_shape or tuple(y.shape) != y_shape:
        raise ValueError(f"h must be {list(h_shape)} and y {list(y_shape)}")
    if m == 0:
        name = f"{prefix}_ffn_swiglu"
        rc = getattr(lib(), name)(gate.data_ptr(), gate_scale.data_ptr(), up.data_ptr(), up_scale.data_ptr(),
                                  down.data_ptr(), down_scale.data_ptr(), d_model, d_ff, x.data_ptr(), h.data_ptr(),
                                  y.data_ptr(), _stream(gate))
    else:
        name = f"{prefix}_ffn_swiglu_small"
        rc = getattr(lib(), name)(gate.data_ptr(), gate_scale.data_ptr(), up.data_ptr(), up_scale.data_ptr(),
                                  down.data_ptr(), down_scale.data_ptr(), d_model, d_ff, x.data_ptr(), m,
                                  h.data_ptr(), y.data_ptr(), _stream(gate))
    _check(name, rc)
    return h, y


def ternary_ffn_swiglu(gate: torch.Tensor, gate_scale: torch.Tensor, up: torch.Tensor, up_scale: torch.Tensor,
                       down: torch.Tensor, down_scale: torch.Tensor, x: torch.Tensor,
                       h: torch.Tensor | None = None, y: torch.Tensor | None = None):
    """Gated feed-forward block: h = fp16(silu(gate x) * up x), y = down h.

    gate, up: packed [d_ff, words_per_row(d_model)]; down: packed [d_model, words_per_row(d_ff)];
    x fp16 [d_model] -> (h fp16 [d_ff], y fp32 [d_model]), or x [m, d_model] with m <= 8 ->
    (h [m, d_ff], y [m, d_model]), each weight read once for all m rows.
    """
    return _ffn_swiglu("ternary", words_per_row, gate, gate_scale, up, up_scale, down, down_scale, x, h, y)


def ternary3_ffn_swiglu(gate: torch.Tensor, gate_scale: torch.Tensor, up: torch.Tensor, up_scale: torch.Tensor,
                        down: torch.Tensor, down_scale: torch.Tensor, x: torch.Tensor,
                        h: torch.Tensor | None = None, y: torch.Tensor | None = None):
    """ternary_ffn_swiglu with the three linears in the 3-bit layout (rows of words_per_row3 words)."""
    return _ffn_swiglu("ternary3", words_per_row3, gate, gate_scale, up, up_scale, down, down_scale, x, h, y)


def q8_row_bytes(k: int) -> int:
    """Bytes of an 8-bit activation row of k codes (64 * ceil(k / 64))."""
    return 0 if k <= 0 else (int(k) + 63) // 64 * 64


# The calls below run for every token, with kernels of a few microseconds, so their checks use the cheapest queries:
# the device index, the raw stream handle (a torch.cuda.Stream object costs as much as a small kernel) and identity
# of types; what fails them is looked at again to say why.


def _call(name: str, fn, index: int, *args) -> None:
    """Call the C entry point fn on the current stream of device `index`, whatever the current device is."""
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        _check(name, rc)


def _on(index: int, t, name: str, dtype: torch.dtype, shape: tuple) -> int:
    """Address of t after checking that it is a contiguous dtype tensor of that shape on device `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on device {index}")


def _matrix(t, name: str, dtype: torch.dtype):
    """Rows, columns and device index of t after checking that it is a contiguous dtype matrix on a GPU."""
    try:
        rows, columns = t.shape
        if t.dtype is dtype and t.is_cuda and t.is_contiguous():
            return rows, columns, t.get_device()
    except (AttributeError, TypeError, ValueError):
        pass
    _dev(t, name, dtype)
    raise ValueError(f"{name} must have two dimensions")


def add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                residual_out: torch.Tensor | None = None, h: torch.Tensor | None = None, q: torch.Tensor | None = None,
                q_scale: torch.Tensor | None = None, want: str | None = None):
    """Residual addition and root-mean-square norm of fp32 rows x [m, k]: (residual_out, h, q, q_scale).

    r = x + residual goes to residual_out, which may be x or residual for an update in place; without
    a residual r is x, which is returned itself unless residual_out is given. h is the normed row in
    fp16 [m, k]; q int8 [m, q8_row_bytes(k)] and q_scale fp32 [m] are the same row in 8 bits. Outputs
    are the tensors given; `want` ("h", "q" or "hq") allocates those of its letters that are not. With
    neither, h is allocated. Outputs not asked for are None.
    """
    m, k, dev = _matrix(x, "x", torch.float32)
    if want is None:
        want = "h" if h is None and q is None and q_scale is None else ""
    elif want not in ("h", "q", "hq"):
        raise ValueError('want must be "h", "q" or "hq"')
    if residual_out is None and residual is not None:
        residual_out = torch.empty_like(x)
    if h is None and "h" in want:
        h = torch.empty((m, k), dtype=torch.float16, device=dev)
    if "q" in want or q is not None or q_scale is not None:
        if q is None:
            q = torch.empty((m, q8_row_bytes(k)), dtype=torch.int8, device=dev)
        if q_scale is None:
            q_scale = torch.empty((m,), dtype=torch.float32, device=dev)
    _call("add_rmsnorm", lib().add_rmsnorm, dev, x.data_ptr(),
          None if residual is None else _on(dev, residual, "residual", torch.float32, (m, k)),
          _on(dev, weight, "weight", torch.float32, (k,)), eps, m, k,
          None if residual_out is None else _on(dev, residual_out, "residual_out", torch.float32, (m, k)),
          None if h is None else _on(dev, h, "h", torch.float16, (m, k)),
          None if q is None else _on(dev, q, "q", torch.int8, (m, q8_row_bytes(k))),
          None if q is None else _on(dev, q_scale, "q_scale", torch.float32, (m,)))
    return x if residual_out is None else residual_out, h, q, q_scale


def quantize_rows(x: torch.Tensor, q: torch.Tensor | None = None, q_scale: torch.Tensor | None = None):
    """8-bit form of fp16 rows x [m, k]: (q int8 [m, q8_row_bytes(k)], q_scale fp32 [m]), x ~ q_scale * q."""
    m, k, dev = _matrix(x, "x", torch.float16)
    if q is None:
        q = torch.empty((m, q8_row_bytes(k)), dtype=torch.int8, device=dev)
    if q_scale is None:
        q_scale = torch.empty((m,), dtype=torch.float32, device=dev)
    _call("quantize_rows", lib().quantize_rows, dev, x.data_ptr(), m, k,
          _on(dev, q, "q", torch.int8, (m, q8_row_bytes(k))), _on(dev, q_scale, "q_scale", torch.float32, (m,)))
    return q, q_scale


def ternary_gemm_i8(packed: torch.Tensor, scale: torch.Tensor, k: int, q: torch.Tensor, q_scale: torch.Tensor,
                    y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[i, r] = q_scale[i] * scale[r] * sum_j c[r, j] * q[i, j], exact sums, any number of rows.

    q int8 [m, q8_row_bytes(k)] and q_scale fp32 [m] as add_rmsnorm and quantize_rows leave them; Y fp32 [m, n].
    """
    n, words, dev = _matrix(packed, "packed", torch.int32)
    m, kp = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 2 else 0, q8_row_bytes(k)
    if words != kp // 16:
        raise ValueError(f"packed must be [n, {kp // 16}] for k={k}")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    _call("ternary_gemm_i8", lib().ternary_gemm_i8, dev, packed.data_ptr(),
          _on(dev, scale, "scale", torch.float32, (n,)), n, k, _on(dev, q, "q", torch.int8, (m, kp)),
          _on(dev, q_scale, "q_scale", torch.float32, (m,)), m,
          _on(dev, y, "y", torch.float32, (m, n)))
    return y


def ternary_swiglu_gate_up_i8(gate: torch.Tensor, gate_scale: torch.Tensor, up: torch.Tensor, up_scale: torch.Tensor,
                              d_model: int, q: torch.Tensor, q_scale: torch.Tensor,
                              h: torch.Tensor | None = None) -> torch.Tensor:
    """h = fp16(silu(gate q) * up q) for 8-bit rows q [m, q8_row_bytes(d_model)]; h fp16 [m, d_ff]."""
    d_ff, words, dev = _matrix(gate, "gate", torch.int32)
    m, kp = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 2 else 0, q8_row_bytes(d_model)
    if words != kp // 16:
        raise ValueError(f"gate and up must be [d_ff, {kp // 16}]")
    if h is None:
        h = torch.empty((m, d_ff), dtype=torch.float16, device=dev)
    _call("ternary_swiglu_gate_up_i8", lib().ternary_swiglu_gate_up_i8, dev, gate.data_ptr(),
          _on(dev, gate_scale, "gate_scale", torch.float32, (d_ff,)),
          _on(dev, up, "up", torch.int32, (d_ff, words)), _on(dev, up_scale, "up_scale", torch.float32, (d_ff,)),
          d_model, d_ff, _on(dev, q, "q", torch.int8, (m, kp)), _on(dev, q_scale, "q_scale", torch.float32, (m,)), m,
          _on(dev, h, "h", torch.float16, (m, d_ff)))
    return h


def lora_workspace(m: int, rank: int, device) -> torch.Tensor:
    """A workspace for lora_add on up to m rows and ranks up to rank (its contents do not matter)."""
    return torch.empty((int(lib().pbg_lora_workspace_bytes(int(m), int(rank))),), dtype=torch.uint8, device=device)


def lora_add(y: torch.Tensor, x: torch.Tensor, ids: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
             scale: torch.Tensor, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out[i] = y[i] + scale[t] * b[t] @ (a[t] @ x[i]) with t = ids[i]; rows with t outside [0, adapters) are copied.

    y, out fp32 [m, n] (out may be y); x fp16 [m, k]; ids int32 [m]; a fp16 [adapters, rank, k];
    b fp16 [adapters, n, rank]; scale fp32 [adapters]; workspace from lora_workspace of as many rows
    and as high a rank, or any larger tensor (a new one is allocated if not given).
    """
    m, n, dev = _matrix(y, "y", torch.float32)
    _dev(a, "a", torch.float16)
    if a.dim() != 3:
        raise ValueError("a must be [adapters, rank, k]")
    adapters, rank, k = a.shape
    if out is None:
        out = torch.empty_like(y)
    if workspace is None:
        workspace = lora_workspace(m, rank, dev)
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on device {dev}")
    _call("lora_add", lib().lora_add, dev, y.data_ptr(), _on(dev, x, "x", torch.float16, (m, k)),
          _on(dev, ids, "ids", torch.int32, (m,)), _on(dev, a, "a", torch.float16, (adapters, rank, k)),
          _on(dev, b, "b", torch.float16, (adapters, n, rank)), _on(dev, scale, "scale", torch.float32, (adapters,)),
          m, n, k, adapters, rank, _on(dev, out, "out", torch.float32, (m, n)), workspace.data_ptr(),
          workspace.nbytes)
    return out


def _masks(index: int, t, m: int) -> int:
    """Address of ancestors, an int64 or uint64 [m] tensor of bit masks."""
    unsigned = isinstance(t, torch.Tensor) and t.dtype is torch.uint64
    return _on(index, t, "ancestors", torch.uint64 if unsigned else torch.int64, (m,))


def _cache(k_cache, v_cache):
    """Pages, key heads, page size, head width and device index of a pair of caches."""
    try:
        pages, kv_heads, page_size, head_dim = k_cache.shape
        fine = k_cache.dtype is torch.float16 and k_cache.is_cuda and k_cache.is_contiguous()
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _dev(k_cache, "k_cache", torch.float16)
        raise ValueError("k_cache must be [pages, kv_heads, page_size, head_dim]")
    dev = k_cache.get_device()
    _on(dev, v_cache, "v_cache", torch.float16, k_cache.shape)
    return pages, kv_heads, page_size, head_dim, dev


def cache_plan(lengths: torch.Tensor, added: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
               free_count: torch.Tensor, page_size: int, pages: int, row_start: torch.Tensor | None = None,
               request: torch.Tensor | None = None, position: torch.Tensor | None = None,
               slot: torch.Tensor | None = None, free_left: torch.Tensor | None = None,
               parents: torch.Tensor | None = None, ancestors: torch.Tensor | None = None, rows: int | None = None):
    """The tables of one step over the paged cache: (row_start, request, position, slot, ancestors, free_left).

    lengths, added int32 [requests]: the tokens that each request has in the cache and the rows that it adds. table
    int32 [requests, width] is read and, for pages that the step opens, written; free_pages int32 [n] is a stack of
    free pages with free_count int32 [1] of them left, free_left int32 [1] what the step leaves. parents int32 [rows]
    makes each request's rows a tree of drafted tokens, of at most 64 (from the 64th on a row has no place: prompts that
    are longer need a call without parents). The step has as many rows as the outputs that
    are given, or `rows`: request, position int32 [rows], slot int64 [rows] (-1 for rows behind the last request),
    row_start int32 [requests + 1], ancestors int64 [rows] (bit masks over the request's rows; allocated for a tree).
    Pages are only taken: those that rows which are not kept opened, and those of requests that end, go back onto the
    stack by the caller before the next step.
    """
    i32, i64 = torch.int32, torch.int64
    requests, width, dev = _matrix(table, "table", i32)
    try:
        m = request.numel() if request is not None else int(rows)
        capacity = free_pages.numel()
    except (AttributeError, TypeError):
        raise ValueError("free_pages must be a tensor, and rows (or the outputs) must be given") from None
    if row_start is None:
        row_start = torch.empty((requests + 1,), dtype=i32, device=dev)
    if request is None:
        request = torch.empty((m,), dtype=i32, device=dev)
    if position is None:
        position = torch.empty((m,), dtype=i32, device=dev)
    if slot is None:
        slot = torch.empty((m,), dtype=i64, device=dev)
    if free_left is None:
        free_left = torch.empty((1,), dtype=i32, device=dev)
    if ancestors is None and parents is not None:
        ancestors = torch.empty((m,), dtype=i64, device=dev)
    _call("cache_plan", lib().cache_plan, dev, _on(dev, lengths, "lengths", i32, (requests,)),
          _on(dev, added, "added", i32, (requests,)), requests, table.data_ptr(), width,
          _on(dev, free_pages, "free_pages", i32, (capacity,)), capacity,
          _on(dev, free_count, "free_count", i32, (1,)), pages, page_size,
          None if parents is None else _on(dev, parents, "parents", i32, (m,)), m,
          _on(dev, row_start, "row_start", i32, (requests + 1,)), _on(dev, request, "request", i32, (m,)),
          _on(dev, position, "position", i32, (m,)), _on(dev, slot, "slot", i64, (m,)),
          None if ancestors is None else _masks(dev, ancestors, m), _on(dev, free_left, "free_left", i32, (1,)))
    return row_start, request, position, slot, ancestors, free_left


def rotary_frequencies(rotary_dim: int, base: float = 1e6, scaling: str | None = None, factor: float = 1.0,
                       original_length: int = 32768, device="cuda"):
    """(inv_freq fp64 [rotary_dim / 2], amplitude) of rotary_qkv: base ** (-2 j / rotary_dim), scaled for contexts
    `factor` times as long.

    scaling: None; "linear", positions divided by the factor; "ntk", the base raised so that the slowest pair turns
    factor times slower and the fastest is kept; "yarn", pairs that turn more than 32 times over original_length tokens
    kept, those that turn less than once divided by the factor, a ramp over the pair's number in between, and an
    amplitude of 1 + 0.1 ln(factor).
    """
    if rotary_dim < 0 or rotary_dim % 2 or not factor >= 1.0:
        raise ValueError("rotary_dim must be even and factor at least 1")
    half = rotary_dim // 2
    amplitude = 1.0
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = [base ** (-2.0 * j / rotary_dim) for j in range(half)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        # number of the pair that turns r times over the original length
        def pair(r):
            return rotary_dim * math.log(original_length / (r * 2.0 * math.pi)) / (2.0 * math.log(base))

        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rotary_dim - 1)
        ramp = [min(max((j - low) / max(high - low, 0.001), 0.0), 1.0) for j in range(half)]
        freq = [f / factor * r + f * (1.0 - r) for f, r in zip(freq, ramp)]
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError('scaling must be None, "linear", "ntk" or "yarn"')
    return torch.tensor(freq, dtype=torch.float64, device=device), amplitude


def rotary_qkv(qkv: torch.Tensor, position: torch.Tensor, slot: torch.Tensor, inv_freq: torch.Tensor | None,
               k_cache: torch.Tensor, v_cache: torch.Tensor, q_weight: torch.Tensor | None = None,
               k_weight: torch.Tensor | None = None, eps: float = 1e-6, amplitude: float = 1.0,
               interleaved: bool = False, q: torch.Tensor | None = None) -> torch.Tensor:
    """Queries fp16 [m, heads, head_dim] of a q|k|v linear's output, with its keys and values written into the cache.

    qkv fp32 [m, (heads + 2 kv_heads) * head_dim]; position int32 [m] and slot int64 [m] from cache_plan; inv_freq
    fp64 [rotary_dim / 2] and amplitude from rotary_frequencies (None: nothing is turned); k_cache, v_cache fp16
    [pages, kv_heads, page_size, head_dim]; q_weight, k_weight fp32 [head_dim] norm each q and k head. Rows with a
    negative position are left out.
    """
    pages, kv_heads, page_size, head_dim, dev = _cache(k_cache, v_cache)
    m, columns, _ = _matrix(qkv, "qkv", torch.float32)
    heads = columns // head_dim - 2 * kv_heads if head_dim else 0
    if heads < 1 or columns != (heads + 2 * kv_heads) * head_dim:
        raise ValueError(f"qkv must be [m, (heads + 2 * {kv_heads}) * {head_dim}]")
    if q is None:
        q = torch.empty((m, heads, head_dim), dtype=torch.float16, device=qkv.device)
    half = 0 if inv_freq is None else inv_freq.numel()
    _call("rotary_qkv", lib().rotary_qkv, dev, _on(dev, qkv, "qkv", torch.float32, (m, columns)),
          _on(dev, position, "position", torch.int32, (m,)), _on(dev, slot, "slot", torch.int64, (m,)),
          _on(dev, inv_freq, "inv_freq", torch.float64, (half,)) if half else None,
          None if q_weight is None else _on(dev, q_weight, "q_weight", torch.float32, (head_dim,)),
          None if k_weight is None else _on(dev, k_weight, "k_weight", torch.float32, (head_dim,)), eps, amplitude,
          int(interleaved), m, heads, kv_heads, head_dim, 2 * half,
          _on(dev, q, "q", torch.float16, (m, heads, head_dim)), k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size)
    return q


def attention_workspace(heads: int, kv_heads: int, head_dim: int, device) -> torch.Tensor:
    """A workspace for tree_attention with heads of these shapes, any number of rows (its contents do not matter)."""
    size = int(lib().pbg_attention_workspace_bytes(int(heads), int(kv_heads), int(head_dim)))
    return torch.empty((size,), dtype=torch.uint8, device=device)


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                   lengths: torch.Tensor, row_start: torch.Tensor, ancestors: torch.Tensor | None = None,
                   scale: float | None = None, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of a step's rows over the paged cache: out fp16 [m, heads, head_dim].

    q as rotary_qkv leaves it; k_cache, v_cache fp16 [pages, kv_heads, page_size, head_dim], which hold the step's own
    keys and values already; table int32 [requests, width]; lengths int32 [requests], the tokens before the step;
    row_start int32 [requests + 1] and ancestors int64 [m] from cache_plan. Each row sees its request's tokens from
    before the step, and of the step's own those of its ancestors, or without ancestors those up to itself. Ancestors
    reach over the first 64 rows of a request: leave them out for longer prompts. scale
    defaults to 1 / sqrt(head_dim). A row that sees nothing is zero; rows behind the last request are left as they were.
    """
    pages, kv_heads, page_size, head_dim, dev = _cache(k_cache, v_cache)
    try:
        m, heads, d = q.shape
        requests, width = table.shape
    except (AttributeError, ValueError):
        raise ValueError("q must be [m, heads, head_dim] and table [requests, width]") from None
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = attention_workspace(heads, kv_heads, head_dim, q.device)
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on device {dev}")
    _call("tree_attention", lib().tree_attention, dev, _on(dev, q, "q", torch.float16, (m, heads, head_dim)),
          k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size,
          _on(dev, table, "table", torch.int32, (requests, width)), width,
          _on(dev, lengths, "lengths", torch.int32, (requests,)),
          _on(dev, row_start, "row_start", torch.int32, (requests + 1,)), requests,
          None if ancestors is None else _masks(dev, ancestors, m), m, heads, kv_heads, head_dim,
          head_dim ** -0.5 if scale is None else scale, _on(dev, out, "out", torch.float16, (m, heads, head_dim)),
          workspace.data_ptr(), workspace.nbytes)
    return out


def logits_workspace(m: int, n: int, device) -> torch.Tensor:
    """A workspace for the greedy token of penalize_logits on [m, n] logits (its contents do not matter)."""
    return torch.empty((int(m) * ((int(n) + LOGITS_SLICE - 1) // LOGITS_SLICE),), dtype=torch.int64, device=device)


def penalize_logits(logits: torch.Tensor, request: torch.Tensor, tokens: torch.Tensor, prompt_length: torch.Tensor,
                    length: torch.Tensor, repetition: torch.Tensor, frequency: torch.Tensor, presence: torch.Tensor,
                    drafts: torch.Tensor | None = None, row_start: torch.Tensor | None = None,
                    ancestors: torch.Tensor | None = None, bias_start: torch.Tensor | None = None,
                    bias_token: torch.Tensor | None = None, bias_value: torch.Tensor | None = None,
                    grammar: torch.Tensor | None = None, grammar_row: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, token: torch.Tensor | None = None,
                    top: torch.Tensor | None = None, workspace: torch.Tensor | None = None, greedy: bool = False):
    """Logits fp32 [m, n] under their requests' settings: (out, token, top).

    request int32 [m]; tokens int32 [requests, width] with length and prompt_length int32 [requests] (all, and those of
    the prompt); repetition, frequency, presence fp32 [requests]. drafts int32 [m], row_start and ancestors (cache_plan)
    add each row's drafted tokens to its output. bias_start int32 [requests + 1], bias_token int32 and bias_value fp32
    [entries] list biases; grammar int32 [states, ceil(n / 32)] holds bit masks of allowed tokens, grammar_row int32 [m]
    each row's state (-1: none). out may be logits itself. With greedy=True or token and top given, token int32 [m]
    and top fp32 [m] are the best token and its value (-1 and -infinity where nothing is allowed).
    """
    m, n, dev = _matrix(logits, "logits", torch.float32)
    i32, f32 = torch.int32, torch.float32
    try:
        requests, width = tokens.shape
    except (AttributeError, ValueError):
        raise ValueError("tokens must be [requests, width]") from None
    if out is None:
        out = torch.empty_like(logits)
    if greedy or token is not None or top is not None:
        if token is None:
            token = torch.empty((m,), dtype=i32, device=logits.device)
        if top is None:
            top = torch.empty((m,), dtype=f32, device=logits.device)
        if workspace is None:
            workspace = logits_workspace(m, n, logits.device)
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on device {dev}")
    entries = 0 if bias_token is None else bias_token.numel()
    if bias_token is not None and entries == 0:
        bias_start = bias_token = bias_value = None
    states = 0 if grammar is None else grammar.shape[0]
    _call("penalize_logits", lib().penalize_logits, dev, logits.data_ptr(), _on(dev, request, "request", i32, (m,)),
          _on(dev, tokens, "tokens", i32, (requests, width)), width,
          _on(dev, prompt_length, "prompt_length", i32, (requests,)), _on(dev, length, "length", i32, (requests,)),
          _on(dev, repetition, "repetition", f32, (requests,)), _on(dev, frequency, "frequency", f32, (requests,)),
          _on(dev, presence, "presence", f32, (requests,)), requests,
          None if drafts is None else _on(dev, drafts, "drafts", i32, (m,)),
          None if row_start is None else _on(dev, row_start, "row_start", i32, (requests + 1,)),
          None if ancestors is None else _masks(dev, ancestors, m),
          None if bias_start is None else _on(dev, bias_start, "bias_start", i32, (requests + 1,)),
          None if bias_token is None else _on(dev, bias_token, "bias_token", i32, (entries,)),
          None if bias_value is None else _on(dev, bias_value, "bias_value", f32, (entries,)), entries,
          None if grammar is None else _on(dev, grammar, "grammar", i32, (states, (n + 31) // 32)),
          None if grammar_row is None else _on(dev, grammar_row, "grammar_row", i32, (m,)), states, m, n,
          _on(dev, out, "out", f32, (m, n)), None if token is None else _on(dev, token, "token", i32, (m,)),
          None if top is None else _on(dev, top, "top", f32, (m,)),
          None if token is None else workspace.data_ptr(), 0 if token is None else workspace.nbytes)
    return out, token, top


def stream_read(src: torch.Tensor, sink: torch.Tensor | None = None) -> torch.Tensor:
    """Read every byte of src once with the GEMVs' loads and fold them by XOR into sink.

    A measurement helper: its time is the streaming-read ceiling for one launch
    moving src.nbytes. sink is int32 [STREAM_READ_SINK_WORDS] (a new zeroed one
    if None); afterwards the XOR of its words, XOR-ed with its XOR before the
    call, is the XOR of all 32-bit words of src.
    """
    if not isinstance(src, torch.Tensor) or not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous CUDA (HIP) tensor")
    if sink is None:
        sink = torch.zeros((STREAM_READ_SINK_WORDS,), dtype=torch.int32, device=src.device)
    _dev(sink, "sink", torch.int32)
    if tuple(sink.shape) != (STREAM_READ_SINK_WORDS,):
        raise ValueError(f"sink must be [{STREAM_READ_SINK_WORDS}]")
    nbytes = src.numel() * src.element_size()
    rc = lib().pbg_stream_read(src.data_ptr(), nbytes, sink.data_ptr(), _stream(src))
    _check("pbg_stream_read", rc)
    return sink
