"""Python binding of libmxmoe (MXFP8 quantisers and dropless grouped GEMMs for MI355X / gfx950).

Argument marshalling only: every step runs in the HIP library.  Tensors are torch tensors on the
current HIP device (bf16 inputs may be given as torch.bfloat16 or as uint16/int16 bit patterns);
outputs are allocated with torch when not passed in.  Calls are asynchronous on torch's current
stream unless `stream` (a torch.cuda.Stream or a raw hipStream_t integer) is given; outputs that a call
allocates then belong to that stream, as inside torch.cuda.stream(stream).

The library must be built (``python -m precision_moe_expert_mx_amd.build``); importing this package
without it raises, and there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

__all__ = [
    "LIB_PATH", "MxMoeError", "lib", "abi_version",
    "mx_colwise_ld_min", "mxmoe_pitch", "mx_colwise_ld", "mxfp4_colwise_ld",
    "mx_quantize_rowwise", "mx_quantize_colwise", "mx_quantize_dual",
    "mx_grouped_gemm_fwd", "mx_grouped_gemm_dgrad", "mx_grouped_gemm_wgrad", "mx_grouped_gemm_fwd_swiglu",
    "mx_quantize_rowwise_tiled", "mx_quantize_colwise_tiled", "mx_quantize_dual_tiled", "mx_grouped_gemm_fwd_tiled",
    "mx_grouped_gemm_fwd_swiglu_tiled", "mx_grouped_gemm_dgrad_tiled", "mx_grouped_gemm_wgrad_tiled",
    "fp8bw_quantize_act_1x128", "fp8bw_quantize_weight_128x128",
    "fp8bw_grouped_gemm_fwd", "fp8bw_grouped_gemm_dgrad", "mxmoe_check_offsets",
    "fp8bw_grouped_gemm_fwd_pow2", "fp8bw_grouped_gemm_dgrad_pow2", "fp8bw_grouped_gemm_wgrad_pow2",
    "fp8bw_colwise_ld_min", "fp8bw_quantize_colwise_128", "fp8bw_grouped_gemm_wgrad",
    "mxfp4_quantize_rowwise", "mxfp4_quantize_colwise", "mxfp4_grouped_gemm_fwd", "mxfp4_grouped_gemm_dgrad",
    "mxfp4_grouped_gemm_wgrad",
    "bf16_grouped_gemm_fwd", "bf16_grouped_gemm_dgrad", "bf16_grouped_gemm_wgrad",
    "int8_quantize_rowwise", "int8_quantize_swiglu_rowwise", "int8_grouped_gemm_fwd",
    "AdamWTable", "adamw_table", "adamw_step", "adamw_dequantize",
    "rmsnorm_fwd", "int8_quantize_rmsnorm_rowwise", "mx_quantize_rmsnorm_rowwise", "rmsnorm_bwd",
    "moe_route_fwd", "moe_sort", "moe_route_sort", "moe_route_bwd",
    "moe_dispatch", "moe_combine_fwd", "moe_combine_bwd",
    "EXPORTED_SYMBOLS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxmoe.so")

MXMOE_F32, MXMOE_BF16 = 0, 1
_STATUS = {0: "OK", 1: "ERR_NULL", 2: "ERR_SHAPE", 3: "ERR_ALIGN", 4: "ERR_DTYPE", 5: "ERR_OFFSETS",
           6: "ERR_HIP", 7: "ERR_UNSUPPORTED"}

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_int = ctypes.c_int
_f64 = ctypes.c_double

# name -> (restype, argtypes); mirrors include/mxmoe.h
_SIGS = {
    "mxmoe_abi_version": (ctypes.c_int, []),
    "mxmoe_last_error": (ctypes.c_char_p, []),
    "mx_colwise_ld_min": (_i64, [_i64, _i32]),
    "mxmoe_pitch": (_i64, [_i64]),
    "mx_quantize_rowwise": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "mx_quantize_colwise": (ctypes.c_int, [_p, _i64, _i64, _p, _i32, _p, _p, _i64, _p]),
    "mx_quantize_dual": (ctypes.c_int, [_p, _i64, _i64, _p, _i64, _p, _i32, _p, _p, _p, _p, _i64, _p]),
    "mx_grouped_gemm_fwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "mx_grouped_gemm_fwd_swiglu": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p,
                                                  _i64, _p]),
    "mx_grouped_gemm_dgrad": (ctypes.c_int, [_p, _p, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "mx_grouped_gemm_wgrad": (ctypes.c_int, [_p, _p, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "fp8bw_quantize_act_1x128": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "fp8bw_quantize_weight_128x128": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p, _p]),
    "fp8bw_grouped_gemm_fwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "fp8bw_grouped_gemm_dgrad": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "fp8bw_colwise_ld_min": (_i64, [_i64, _i32]),
    "mxfp4_quantize_rowwise": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "mxfp4_quantize_colwise": (ctypes.c_int, [_p, _i64, _i64, _p, _i32, _p, _p, _i64, _p]),
    "mxfp4_grouped_gemm_fwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "mxfp4_grouped_gemm_dgrad": (ctypes.c_int, [_p, _p, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int,
                                                _p]),
    "mxfp4_grouped_gemm_wgrad": (ctypes.c_int, [_p, _p, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int,
                                                _p]),
    "fp8bw_quantize_colwise_128": (ctypes.c_int, [_p, _i64, _i64, _p, _i32, _p, _p, _i64, _p]),
    "fp8bw_quantize_act_1x128_pow2": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "fp8bw_quantize_weight_128x128_pow2": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p, _p]),
    "fp8bw_quantize_colwise_128_pow2": (ctypes.c_int, [_p, _i64, _i64, _p, _i32, _p, _p, _i64, _p]),
    "fp8bw_grouped_gemm_wgrad": (ctypes.c_int, [_p, _p, _p, _p, _i64, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int,
                                                _p]),
    "mxmoe_check_offsets": (ctypes.c_int, [_p, _i32, _i64, _p]),
    "bf16_grouped_gemm_fwd": (ctypes.c_int, [_p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "bf16_grouped_gemm_dgrad": (ctypes.c_int, [_p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "bf16_grouped_gemm_wgrad": (ctypes.c_int, [_p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "int8_quantize_rowwise": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "int8_quantize_swiglu_rowwise": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "int8_grouped_gemm_fwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, ctypes.c_int, _p]),
    "adamw_step": (ctypes.c_int, [_p, _i32, ctypes.c_int, _i32, _p, _p]),
    "adamw_dequantize": (ctypes.c_int, [_p, _p, _i64, _i32, _p, ctypes.c_int, _p]),
    "rmsnorm_fwd": (_int, [_p, _int, _p, _int, _p, _int, _i64, _i64, _f64, _p, _int, _p, _p]),
    "int8_quantize_rmsnorm_rowwise": (_int, [_p, _int, _p, _int, _p, _int, _i64, _i64, _f64, _p, _p, _p, _p, _p]),
    "mx_quantize_rmsnorm_rowwise": (_int, [_p, _int, _p, _int, _p, _int, _i64, _i64, _f64, _p, _p, _p, _p, _p]),
    "rmsnorm_bwd_workspace": (_i64, [_i64, _i64]),
    "rmsnorm_bwd": (_int, [_p, _int, _p, _int, _p, _int, _p, _i64, _i64, _f64, _p, _p, _p, _p]),
    "moe_route_fwd": (_int, [_p, _int, _p, _p, _i64, _i32, _i32, _int, _i32, _i32, _i32, _i32, _f64, _p, _p, _p]),
    "moe_sort_workspace": (_i64, [_i64, _i32]),
    "moe_sort": (_int, [_p, _i64, _i32, _i32, _i32, _p, _p, _p, _p, _p]),
    "moe_route_sort": (_int, [_p, _int, _p, _p, _i64, _i32, _i32, _int, _i32, _i32, _i32, _i32, _f64, _p, _p, _i32, _i32,
                              _p, _p, _p, _p, _p]),
    "moe_route_bwd": (_int, [_p, _p, _p, _int, _i64, _i32, _i32, _int, _i32, _f64, _p, _p]),
    "moe_dispatch": (_int, [_p, _i64, _p, _i64, _p, _i64, _i32, _i64, _p, _p, _p]),
    "moe_combine_fwd": (_int, [_p, _int, _p, _p, _p, _int, _i64, _i32, _i64, _i64, _p, _int, _p]),
    "moe_combine_bwd": (_int, [_p, _int, _p, _p, _p, _int, _i64, _i32, _i64, _i64, _p, _p, _p]),
}
# the 128-byte tiled layouts: the same arguments as the row-major entry points
for _n in ("mx_quantize_rowwise", "mx_quantize_colwise", "mx_quantize_dual", "mx_grouped_gemm_fwd",
           "mx_grouped_gemm_fwd_swiglu", "mx_grouped_gemm_dgrad", "mx_grouped_gemm_wgrad"):
    _SIGS[_n + "_tiled"] = _SIGS[_n]
# blockwise forward / dgrad for power-of-two scales (on the MX kernel): the same arguments
_SIGS["fp8bw_grouped_gemm_fwd_pow2"] = _SIGS["fp8bw_grouped_gemm_fwd"]
_SIGS["fp8bw_grouped_gemm_dgrad_pow2"] = _SIGS["fp8bw_grouped_gemm_dgrad"]
_SIGS["fp8bw_grouped_gemm_wgrad_pow2"] = _SIGS["fp8bw_grouped_gemm_wgrad"]
# the full-rate FP8 operand feed: the same arguments as the precise entry points
for _n in ("fp8bw_grouped_gemm_fwd_pow2", "fp8bw_grouped_gemm_dgrad_pow2", "fp8bw_grouped_gemm_wgrad_pow2", "mx_grouped_gemm_fwd", "mx_grouped_gemm_dgrad", "mx_grouped_gemm_wgrad", "fp8bw_grouped_gemm_fwd",
           "fp8bw_grouped_gemm_dgrad", "fp8bw_grouped_gemm_wgrad", "mx_grouped_gemm_fwd_tiled",
           "mx_grouped_gemm_dgrad_tiled", "mx_grouped_gemm_wgrad_tiled"):
    _SIGS[_n + "_fp8feed"] = _SIGS[_n]
EXPORTED_SYMBOLS = tuple(_SIGS)


class MxMoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmxmoe (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m precision_moe_expert_mx_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MxMoeError(fn, status, lib().mxmoe_last_error().decode(errors="replace"))


def abi_version() -> int:
    return lib().mxmoe_abi_version()


def mx_colwise_ld_min(M: int, G: int) -> int:
    return lib().mx_colwise_ld_min(int(M), int(G))


def mxmoe_pitch(min_ld: int) -> int:
    """The recommended row pitch >= min_ld for a column-wise output (avoids slow pitches)."""
    return lib().mxmoe_pitch(int(min_ld))


def mxfp4_colwise_ld(M: int, G: Optional[int] = None) -> int:
    """Default leading dimension (elements) of a column-wise MXFP4 output: qT rows hold ld / 2 bytes, so
    the recommended pitch applies to the byte count."""
    need = mx_colwise_ld_min(M, G) if G is not None else 32 * ((int(M) + 31) // 32)
    return 2 * mxmoe_pitch(need // 2)


def mx_colwise_ld(M: int, G: Optional[int] = None) -> int:
    """Default leading dimension of a column-wise MX output of R = M rows: the recommended pitch for G
    groups (routing offsets), or for one group of M rows when G is None (a weight viewed as [G*N, K])."""
    need = mx_colwise_ld_min(M, G) if G is not None else 32 * ((int(M) + 31) // 32)
    return mxmoe_pitch(need)


# ---------------------------------------------------------------- torch plumbing
@functools.lru_cache(None)
def _torch():
    import torch
    return torch


def _stream_handle(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _bf16_bits(x):
    torch = _torch()
    if x.dtype == torch.bfloat16 or x.dtype in (torch.int16, torch.uint16):
        return x
    raise TypeError(f"expected bfloat16 (or its 16-bit pattern), got {x.dtype}")


def _empty(shape, dtype, like, stream=None):
    """An output of a call on `stream`, from that stream's memory: the current stream may still be using blocks
    that were freed on it."""
    torch = _torch()
    if stream is not None and like.is_cuda:
        handle = _stream_handle(stream)
        if handle != torch._C._cuda_getCurrentRawStream(like.get_device()):
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(handle, like.device) if handle else torch.cuda.default_stream(like.device)
            with torch.cuda.stream(stream):
                return torch.empty(shape, dtype=dtype, device=like.device)
    return torch.empty(shape, dtype=dtype, device=like.device)


@functools.lru_cache(None)
def _out_dtype(dt: str):
    torch = _torch()
    if dt == "f32":
        return torch.float32, MXMOE_F32
    if dt == "bf16":
        return torch.bfloat16, MXMOE_BF16
    raise ValueError(dt)


def _gemm(name: str, fast: bool):
    """The entry point of a GEMM: the precise feed, or its full-rate FP8 feed (`name`_fp8feed)."""
    return (name + "_fp8feed" if fast else name), getattr(lib(), name + "_fp8feed" if fast else name)


def _call(entry, *args):
    name, f = entry
    return name, f(*args)


# ---------------------------------------------------------------- MX quantisers
def _rowwise_scales_out(R, C, tiled, like, stream):
    """A row-wise copy's scale buffer: [R, C / 32], or [C / 128, R, 4] in the tiled layout."""
    torch = _torch()
    return _empty((C // 128, R, 4) if tiled else (R, C // 32), torch.uint8, like, stream)


def _rowwise(name, tiled, x, q, s, stream):
    torch = _torch()
    x = _bf16_bits(x)
    R, C = x.shape
    q = _empty((R, C), torch.uint8, x, stream) if q is None else q
    s = _rowwise_scales_out(R, C, tiled, x, stream) if s is None else s
    _check(name, getattr(lib(), name)(_ptr(x), R, C, _ptr(q), _ptr(s), _stream_handle(stream)))
    return q, s


def mx_quantize_rowwise(x, q=None, s=None, stream=None) -> Tuple[object, object]:
    """x bf16 [R, C] -> (q uint8 [R, C], s uint8 [R, C/32])."""
    return _rowwise("mx_quantize_rowwise", False, x, q, s, stream)


def mx_quantize_rowwise_tiled(x, q=None, s=None, stream=None) -> Tuple[object, object]:
    """As mx_quantize_rowwise with the scales in the tiled layout: s uint8 [C/128, R, 4] (C % 128 == 0)."""
    return _rowwise("mx_quantize_rowwise_tiled", True, x, q, s, stream)


def _colwise_out(C, ld, tiled, like, stream):
    """A column-wise code buffer: [C, ld] row-major, or [ld / 128, C, 128] in the tiled layout."""
    torch = _torch()
    return _empty((ld // 128, C, 128) if tiled else (C, ld), torch.uint8, like, stream)


def _colwise_scales_out(C, ld, tiled, like, stream):
    """Its scale buffer: [C, ld / 32] row-major, or [ld / 128, C, 4] in the tiled layout."""
    torch = _torch()
    return _empty((ld // 128, C, 4) if tiled else (C, ld // 32), torch.uint8, like, stream)


def _colwise(name, tiled, x, offs, G, ld, qT, sT, stream):
    torch = _torch()
    x = _bf16_bits(x)
    R, C = x.shape
    if offs is not None:
        G = offs.numel() - 1
    if ld is None:
        ld = mx_colwise_ld(R, G if offs is not None else None)
    qT = _colwise_out(C, ld, tiled, x, stream) if qT is None else qT
    sT = _colwise_scales_out(C, ld, tiled, x, stream) if sT is None else sT
    _check(name, getattr(lib(), name)(_ptr(x), R, C, _ptr(offs), G, _ptr(qT), _ptr(sT), ld, _stream_handle(stream)))
    return qT, sT


def mx_quantize_colwise(x, offs=None, G: int = 1, ld: Optional[int] = None, qT=None, sT=None, stream=None):
    """x bf16 [R, C] -> (qT uint8 [C, ld], sT uint8 [C, ld/32]); offs int32 [G+1] device or None."""
    return _colwise("mx_quantize_colwise", False, x, offs, G, ld, qT, sT, stream)


def mx_quantize_colwise_tiled(x, offs=None, G: int = 1, ld: Optional[int] = None, qT=None, sT=None, stream=None):
    """As mx_quantize_colwise in the 128-byte tiled layout: qT uint8 [ld/128, C, 128], sT [ld/128, C, 4]."""
    return _colwise("mx_quantize_colwise_tiled", True, x, offs, G, ld, qT, sT, stream)


def _dual(name, tiled, x, offs, G, ld, row_idx, q, s, qT, sT, stream):
    torch = _torch()
    x = _bf16_bits(x)
    R_src, C = x.shape
    R = row_idx.numel() if row_idx is not None else R_src
    if offs is not None:
        G = offs.numel() - 1
    if ld is None:
        ld = mx_colwise_ld(R, G if offs is not None else None)
    q = _empty((R, C), torch.uint8, x, stream) if q is None else q
    s = _rowwise_scales_out(R, C, tiled, x, stream) if s is None else s
    qT = _colwise_out(C, ld, tiled, x, stream) if qT is None else qT
    sT = _colwise_scales_out(C, ld, tiled, x, stream) if sT is None else sT
    _check(name, getattr(lib(), name)(_ptr(x), R, C, _ptr(row_idx), R_src, _ptr(offs), G, _ptr(q), _ptr(s), _ptr(qT),
                                      _ptr(sT), ld, _stream_handle(stream)))
    return q, s, qT, sT


def mx_quantize_dual(x, offs=None, G: int = 1, ld: Optional[int] = None, row_idx=None, q=None, s=None, qT=None,
                     sT=None, stream=None):
    """Row-wise and column-wise MX layouts from one read of x.

    x bf16 [R_src, C]; row_idx int32 [R] (routed row r reads x[row_idx[r]]) or None (R = R_src).
    Returns (q [R, C], s [R, C/32], qT [C, ld], sT [C, ld/32]), all uint8."""
    return _dual("mx_quantize_dual", False, x, offs, G, ld, row_idx, q, s, qT, sT, stream)


def mx_quantize_dual_tiled(x, offs=None, G: int = 1, ld: Optional[int] = None, row_idx=None, q=None, s=None,
                           qT=None, sT=None, stream=None):
    """As mx_quantize_dual in the 128-byte tiled layouts: qT [ld/128, C, 128], sT [ld/128, C, 4] and
    s [C/128, R, 4] (C % 128 == 0)."""
    return _dual("mx_quantize_dual_tiled", True, x, offs, G, ld, row_idx, q, s, qT, sT, stream)


# ---------------------------------------------------------------- MX grouped GEMMs
def _fwd(name, qx, sx, qw, sw, offs, N, out_dtype, y, stream, fast):
    M, K = qx.shape
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    y = _empty((M, N), tdt, qx, stream) if y is None else y
    _check(*_call(_gemm(name, fast), _ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(offs), G, M, N, K, _ptr(y), cdt,
                  _stream_handle(stream)))
    return y


def mx_grouped_gemm_fwd(qx, sx, qw, sw, offs, N: int, out_dtype: str = "f32", y=None, stream=None, fast: bool = False):
    """Y [M, N] = per-expert X_g W_g^T from row-wise MX operands (qw: [G*N, K])."""
    return _fwd("mx_grouped_gemm_fwd", qx, sx, qw, sw, offs, N, out_dtype, y, stream, fast)


def mx_grouped_gemm_fwd_tiled(qx, sx, qw, sw, offs, N: int, out_dtype: str = "f32", y=None, stream=None,
                              fast: bool = False):
    """As mx_grouped_gemm_fwd with the scales in the tiled layout (sx [K/128, M, 4], sw [K/128, G*N, 4])."""
    return _fwd("mx_grouped_gemm_fwd_tiled", qx, sx, qw, sw, offs, N, out_dtype, y, stream, fast)


def _swiglu(name, tiled, qx, sx, qw, sw, offs, N, y, qh, sh, h, with_h, colwise, ldh, qhT, shT, stream):
    torch = _torch()
    M, K = qx.shape
    G = offs.numel() - 1
    H = N // 2
    y = _empty((M, N), torch.bfloat16, qx, stream) if y is None else y
    qh = _empty((M, H), torch.uint8, qx, stream) if qh is None else qh
    sh = _rowwise_scales_out(M, H, tiled, qx, stream) if sh is None else sh
    if with_h and h is None:
        h = _empty((M, H), torch.float32, qx, stream)
    if colwise or tiled or qhT is not None:
        if qhT is not None:
            ldh = qhT.shape[0] * 128 if tiled else qhT.shape[1]
        elif ldh is None:
            ldh = mx_colwise_ld(M, G)
        qhT = _colwise_out(H, ldh, tiled, qx, stream) if qhT is None else qhT
        shT = _colwise_scales_out(H, ldh, tiled, qx, stream) if shT is None else shT
    _check(name, getattr(lib(), name)(
        _ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(offs), G, M, N, K, _ptr(y), _ptr(qh), _ptr(sh), _ptr(h),
        _ptr(qhT), _ptr(shT), int(ldh or 0), _stream_handle(stream)))
    out = (y, qh, sh) + ((qhT, shT) if qhT is not None else ())
    return out if h is None else out + (h,)


def mx_grouped_gemm_fwd_swiglu(qx, sx, qw, sw, offs, N: int, y=None, qh=None, sh=None, h=None,
                               with_h: bool = False, colwise: bool = False, ldh: Optional[int] = None, qhT=None,
                               shT=None, stream=None):
    """Forward of the gate+up GEMM (W rows: gate then up of each expert, N = 2H) with SwiGLU and the
    MX quantisation of H in the epilogue.  Returns (y bf16 [M, N], qh [M, H], sh [M, H/32]); with
    colwise (or qhT given) also H column-wise (qhT [H, ldh], shT [H, ldh/32], ldh by default the
    recommended pitch for the routing offsets); with with_h (or h given) H in fp32 [M, H] last."""
    return _swiglu("mx_grouped_gemm_fwd_swiglu", False, qx, sx, qw, sw, offs, N, y, qh, sh, h, with_h, colwise, ldh,
                   qhT, shT, stream)


def mx_grouped_gemm_fwd_swiglu_tiled(qx, sx, qw, sw, offs, N: int, y=None, qh=None, sh=None, h=None,
                                     with_h: bool = False, ldh: Optional[int] = None, qhT=None, shT=None,
                                     stream=None):
    """As mx_grouped_gemm_fwd_swiglu in the 128-byte tiled layouts: sx [K/128, M, 4] and sw [K/128, G*N, 4]
    in; sh [H/128, M, 4], qhT [ldh/128, H, 128], shT [ldh/128, H, 4] out (H always column-wise too).
    Returns (y, qh, sh, qhT, shT[, h])."""
    return _swiglu("mx_grouped_gemm_fwd_swiglu_tiled", True, qx, sx, qw, sw, offs, N, y, qh, sh, h, with_h, True,
                   ldh, qhT, shT, stream)


def mx_grouped_gemm_dgrad(qdy, sdy, qwT, swT, offs, K: int, out_dtype: str = "f32", dx=None, stream=None, fast: bool = False):
    """dX [M, K] = per-expert dY_g W_g from row-wise dY and column-wise W ([K, ldw])."""
    return _dgrad("mx_grouped_gemm_dgrad", qwT.shape[1], qdy, sdy, qwT, swT, offs, K, out_dtype, dx, stream, fast)


def mx_grouped_gemm_dgrad_tiled(qdy, sdy, qwT, swT, offs, K: int, out_dtype: str = "f32", dx=None, stream=None,
                                fast: bool = False):
    """As mx_grouped_gemm_dgrad in the 128-byte tiled layouts: sdy [N/128, M, 4], qwT [ldw/128, K, 128],
    swT [ldw/128, K, 4]."""
    return _dgrad("mx_grouped_gemm_dgrad_tiled", qwT.shape[0] * 128, qdy, sdy, qwT, swT, offs, K, out_dtype, dx,
                  stream, fast)


def _dgrad(name, ldw, qdy, sdy, qwT, swT, offs, K, out_dtype, dx, stream, fast):
    M, N = qdy.shape
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    dx = _empty((M, K), tdt, qdy, stream) if dx is None else dx
    _check(*_call(_gemm(name, fast), _ptr(qdy), _ptr(sdy), _ptr(qwT), _ptr(swT), ldw, _ptr(offs), G, M, N, K,
                  _ptr(dx), cdt, _stream_handle(stream)))
    return dx


def mx_grouped_gemm_wgrad(qdyT, sdyT, qxT, sxT, offs, M: int, out_dtype: str = "f32", dw=None, stream=None, fast: bool = False):
    """dW [G, N, K] = per-expert dY_g^T X_g from column-wise dY ([N, ld]) and X ([K, ld])."""
    N, ld = qdyT.shape
    return _wgrad("mx_grouped_gemm_wgrad", N, ld, qxT.shape[0], qdyT, sdyT, qxT, sxT, offs, M, out_dtype, dw, stream,
                  fast)


def mx_grouped_gemm_wgrad_tiled(qdyT, sdyT, qxT, sxT, offs, M: int, out_dtype: str = "f32", dw=None, stream=None,
                                fast: bool = False):
    """As mx_grouped_gemm_wgrad with qdyT, sdyT / qxT, sxT in the 128-byte tiled layout
    ([ld/128, N, 128], [ld/128, N, 4] / [ld/128, K, 128], [ld/128, K, 4])."""
    return _wgrad("mx_grouped_gemm_wgrad_tiled", qdyT.shape[1], qdyT.shape[0] * 128, qxT.shape[1], qdyT, sdyT, qxT,
                  sxT, offs, M, out_dtype, dw, stream, fast)


def _wgrad(name, N, ld, K, qdyT, sdyT, qxT, sxT, offs, M, out_dtype, dw, stream, fast):
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    dw = _empty((G, N, K), tdt, qdyT, stream) if dw is None else dw
    _check(*_call(_gemm(name, fast), _ptr(qdyT), _ptr(sdyT), _ptr(qxT), _ptr(sxT), ld, _ptr(offs), G, M, N, K,
                  _ptr(dw), cdt, _stream_handle(stream)))
    return dw


# ---------------------------------------------------------------- MXFP4
def mxfp4_quantize_rowwise(x, q=None, s=None, stream=None):
    """x bf16 [R, C] -> (q uint8 [R, C/2] packed E2M1, s uint8 [R, C/32])."""
    torch = _torch()
    x = _bf16_bits(x)
    R, C = x.shape
    q = _empty((R, C // 2), torch.uint8, x, stream) if q is None else q
    s = _empty((R, C // 32), torch.uint8, x, stream) if s is None else s
    _check("mxfp4_quantize_rowwise", lib().mxfp4_quantize_rowwise(_ptr(x), R, C, _ptr(q), _ptr(s),
                                                                  _stream_handle(stream)))
    return q, s


def mxfp4_quantize_colwise(x, offs=None, G: int = 1, ld: Optional[int] = None, qT=None, sT=None, stream=None):
    """x bf16 [R, C] -> (qT uint8 [C, ld/2] packed E2M1, sT uint8 [C, ld/32])."""
    torch = _torch()
    x = _bf16_bits(x)
    R, C = x.shape
    if offs is not None:
        G = offs.numel() - 1
    if ld is None:
        ld = mxfp4_colwise_ld(R, G if offs is not None else None)
    qT = _empty((C, ld // 2), torch.uint8, x, stream) if qT is None else qT
    sT = _empty((C, ld // 32), torch.uint8, x, stream) if sT is None else sT
    _check("mxfp4_quantize_colwise", lib().mxfp4_quantize_colwise(_ptr(x), R, C, _ptr(offs), G, _ptr(qT), _ptr(sT),
                                                                  ld, _stream_handle(stream)))
    return qT, sT


def mxfp4_grouped_gemm_fwd(qx, sx, qw, sw, offs, N: int, out_dtype: str = "f32", y=None, stream=None):
    """Y [M, N] from row-wise MXFP4 X (qx [M, K/2]) and W (qw [G*N, K/2])."""
    M, K = qx.shape[0], 2 * qx.shape[1]
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    y = _empty((M, N), tdt, qx, stream) if y is None else y
    _check("mxfp4_grouped_gemm_fwd", lib().mxfp4_grouped_gemm_fwd(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(offs),
                                                                  G, M, N, K, _ptr(y), cdt, _stream_handle(stream)))
    return y


def mxfp4_grouped_gemm_dgrad(qdy, sdy, qwT, swT, offs, K: int, out_dtype: str = "f32", dx=None, stream=None):
    """dX [M, K] from row-wise MXFP4 dY (qdy [M, N/2]) and column-wise W (qwT [K, ldw/2])."""
    M, N = qdy.shape[0], 2 * qdy.shape[1]
    ldw = 2 * qwT.shape[1]
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    dx = _empty((M, K), tdt, qdy, stream) if dx is None else dx
    _check("mxfp4_grouped_gemm_dgrad", lib().mxfp4_grouped_gemm_dgrad(_ptr(qdy), _ptr(sdy), _ptr(qwT), _ptr(swT), ldw,
                                                                      _ptr(offs), G, M, N, K, _ptr(dx), cdt,
                                                                      _stream_handle(stream)))
    return dx


def mxfp4_grouped_gemm_wgrad(qdyT, sdyT, qxT, sxT, offs, M: int, out_dtype: str = "f32", dw=None, stream=None):
    """dW [G, N, K] from column-wise MXFP4 dY (qdyT [N, ld/2]) and X (qxT [K, ld/2])."""
    N, ld = qdyT.shape[0], 2 * qdyT.shape[1]
    K = qxT.shape[0]
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    dw = _empty((G, N, K), tdt, qdyT, stream) if dw is None else dw
    _check("mxfp4_grouped_gemm_wgrad", lib().mxfp4_grouped_gemm_wgrad(_ptr(qdyT), _ptr(sdyT), _ptr(qxT), _ptr(sxT), ld,
                                                                      _ptr(offs), G, M, N, K, _ptr(dw), cdt,
                                                                      _stream_handle(stream)))
    return dw


# ---------------------------------------------------------------- blockwise FP8
def fp8bw_quantize_act_1x128(x, q=None, s=None, stream=None, pow2: bool = False):
    """x bf16 [R, C] -> (q [R, C], s f32 [R, C/128]); pow2 selects the power-of-two scale mode."""
    torch = _torch()
    x = _bf16_bits(x)
    R, C = x.shape
    q = _empty((R, C), torch.uint8, x, stream) if q is None else q
    s = _empty((R, C // 128), torch.float32, x, stream) if s is None else s
    fn = "fp8bw_quantize_act_1x128" + ("_pow2" if pow2 else "")
    _check(fn, getattr(lib(), fn)(_ptr(x), R, C, _ptr(q), _ptr(s), _stream_handle(stream)))
    return q, s


def fp8bw_quantize_weight_128x128(w, q=None, s=None, qT=None, transposed: bool = False, stream=None,
                                  pow2: bool = False):
    """w bf16 [R, C] -> (q [R, C], s f32 [R/128, C/128]) or, with transposed=True (or qT given),
    (q, s, qT [C, R]) where qT is the dgrad operand; pow2 selects the power-of-two scale mode."""
    torch = _torch()
    w = _bf16_bits(w)
    R, C = w.shape
    q = _empty((R, C), torch.uint8, w, stream) if q is None else q
    s = _empty((R // 128, C // 128), torch.float32, w, stream) if s is None else s
    if transposed and qT is None:
        qT = _empty((C, R), torch.uint8, w, stream)
    fn = "fp8bw_quantize_weight_128x128" + ("_pow2" if pow2 else "")
    _check(fn, getattr(lib(), fn)(_ptr(w), R, C, _ptr(q), _ptr(s), _ptr(qT), _stream_handle(stream)))
    return (q, s) if qT is None else (q, s, qT)


def _bw_fwd(name, qx, sx, qw, sw, offs, N, out_dtype, y, stream, fast):
    M, K = qx.shape
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    y = _empty((M, N), tdt, qx, stream) if y is None else y
    _check(*_call(_gemm(name, fast), _ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(offs), G, M, N, K, _ptr(y), cdt,
                  _stream_handle(stream)))
    return y


def _bw_dgrad(name, qdy, sdy, qwT, sw, offs, K, out_dtype, dx, stream, fast):
    M, N = qdy.shape
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    dx = _empty((M, K), tdt, qdy, stream) if dx is None else dx
    _check(*_call(_gemm(name, fast), _ptr(qdy), _ptr(sdy), _ptr(qwT), _ptr(sw), _ptr(offs), G, M, N, K, _ptr(dx),
                  cdt, _stream_handle(stream)))
    return dx


def fp8bw_grouped_gemm_fwd(qx, sx, qw, sw, offs, N: int, out_dtype: str = "f32", y=None, stream=None, fast: bool = False):
    """Y [M, N] from blockwise X (1x128 tiles) and W (128x128 blocks), promoted per 128-slice."""
    return _bw_fwd("fp8bw_grouped_gemm_fwd", qx, sx, qw, sw, offs, N, out_dtype, y, stream, fast)


def fp8bw_grouped_gemm_dgrad(qdy, sdy, qwT, sw, offs, K: int, out_dtype: str = "f32", dx=None, stream=None,
                             fast: bool = False):
    """dX [M, K] from blockwise dY (1x128 along N) and the transposed weight copy qwT [K, G*N]."""
    return _bw_dgrad("fp8bw_grouped_gemm_dgrad", qdy, sdy, qwT, sw, offs, K, out_dtype, dx, stream, fast)


def fp8bw_grouped_gemm_fwd_pow2(qx, sx, qw, sw, offs, N: int, out_dtype: str = "f32", y=None, stream=None,
                                fast: bool = False):
    """fp8bw_grouped_gemm_fwd for power-of-two scales (the _pow2 quantisers' output), on the MX kernel."""
    return _bw_fwd("fp8bw_grouped_gemm_fwd_pow2", qx, sx, qw, sw, offs, N, out_dtype, y, stream, fast)


def fp8bw_grouped_gemm_dgrad_pow2(qdy, sdy, qwT, sw, offs, K: int, out_dtype: str = "f32", dx=None, stream=None,
                                  fast: bool = False):
    """fp8bw_grouped_gemm_dgrad for power-of-two scales (the _pow2 quantisers' output), on the MX kernel."""
    return _bw_dgrad("fp8bw_grouped_gemm_dgrad_pow2", qdy, sdy, qwT, sw, offs, K, out_dtype, dx, stream, fast)


def fp8bw_colwise_ld_min(M: int, G: int) -> int:
    """Smallest leading dimension of the column-wise blockwise layout (host arithmetic)."""
    return int(lib().fp8bw_colwise_ld_min(M, G))


def fp8bw_quantize_colwise_128(x, offs=None, G: int = 1, ld: Optional[int] = None, qT=None, sT=None, stream=None,
                               pow2: bool = False):
    """x bf16 [R, C] -> (qT uint8 [C, ld], sT float32 [C, ld/128]): 128-row blocks restarting per group;
    pow2 selects the power-of-two scale mode."""
    torch = _torch()
    x = _bf16_bits(x)
    R, C = x.shape
    if offs is not None:
        G = offs.numel() - 1
    if ld is None:
        ld = fp8bw_colwise_ld_min(R, G) if offs is not None else 128 * ((R + 127) // 128)
    qT = _empty((C, ld), torch.uint8, x, stream) if qT is None else qT
    sT = _empty((C, ld // 128), torch.float32, x, stream) if sT is None else sT
    fn = "fp8bw_quantize_colwise_128" + ("_pow2" if pow2 else "")
    _check(fn, getattr(lib(), fn)(_ptr(x), R, C, _ptr(offs), G, _ptr(qT), _ptr(sT), ld, _stream_handle(stream)))
    return qT, sT


def _bw_wgrad(name, qdyT, sdyT, qxT, sxT, offs, M, out_dtype, dw, stream, fast):
    N, ld = qdyT.shape
    K = qxT.shape[0]
    G = offs.numel() - 1
    tdt, cdt = _out_dtype(out_dtype)
    dw = _empty((G, N, K), tdt, qdyT, stream) if dw is None else dw
    _check(*_call(_gemm(name, fast), _ptr(qdyT), _ptr(sdyT), _ptr(qxT), _ptr(sxT), ld, _ptr(offs), G, M, N, K,
                  _ptr(dw), cdt, _stream_handle(stream)))
    return dw


def fp8bw_grouped_gemm_wgrad(qdyT, sdyT, qxT, sxT, offs, M: int, out_dtype: str = "f32", dw=None, stream=None,
                             fast: bool = False):
    """dW [G, N, K] from the column-wise blockwise copies of dY [N, ld] and X [K, ld]."""
    return _bw_wgrad("fp8bw_grouped_gemm_wgrad", qdyT, sdyT, qxT, sxT, offs, M, out_dtype, dw, stream, fast)


def fp8bw_grouped_gemm_wgrad_pow2(qdyT, sdyT, qxT, sxT, offs, M: int, out_dtype: str = "f32", dw=None, stream=None,
                                  fast: bool = False):
    """fp8bw_grouped_gemm_wgrad for power-of-two scales (the _pow2 quantisers' output), on the MX kernel."""
    return _bw_wgrad("fp8bw_grouped_gemm_wgrad_pow2", qdyT, sdyT, qxT, sxT, offs, M, out_dtype, dw, stream, fast)


def mxmoe_check_offsets(offs, M: int, stream=None) -> None:
    G = offs.numel() - 1
    _check("mxmoe_check_offsets", lib().mxmoe_check_offsets(_ptr(offs), G, M, _stream_handle(stream)))


# ---------------------------------------------------------------- plain operands (bf16, int8)
def _run(name, tensors, stream, *args):
    """Launch entry point `name` on the tensors' device (they may live on another one than the current) and on
    that device's current stream unless one is given; the stream is the last argument."""
    index = tensors[0].get_device()
    if index < 0:
        raise ValueError("tensors must be on the GPU")
    for t in tensors:
        if t.get_device() != index:
            raise ValueError(f"tensors must be on one GPU, got {tensors[0].device} and {t.device}")
    _C = _torch()._C
    if _C._cuda_getDevice() != index:
        with _torch().cuda.device(index):
            return _run(name, tensors, stream, *args)
    if stream is None:
        stream = _C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    status = (_entries.get(name) or _entry(name))(*args, stream)
    if status:
        _check(name, status)


_entries = {}


def _entry(name):
    """Entry point `name` of the library, looked up once."""
    return _entries.setdefault(name, getattr(lib(), name))


def _out(t, name, shape, dtype, like, stream):
    """An output: the tensor given, checked, or a new one."""
    if t is not None:
        _want(name, t, (dtype,), shape)
        return t
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    return _empty(shape, dtype, like, stream)


def _want(name, t, dtypes, shape):
    """A tensor argument is contiguous, of one of `dtypes` and of the shape (None: any size), or a clear error
    says what it is not."""
    if t.shape == shape and t.dtype in dtypes and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name}: expected shape {tuple('any' if w is None else w for w in shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")


@functools.lru_cache(None)
def _bf16_types():
    torch = _torch()
    return (torch.bfloat16, torch.int16, torch.uint16)


def _groups(offs):
    n = offs.numel()
    _want("offs", offs, (_torch().int32,), (n,))
    if n < 2:
        raise ValueError("offs: expected G + 1 >= 2 entries")
    return n - 1


def _rows(name, x, dtypes):
    """The shape of a matrix argument."""
    shape = x.shape
    _want(name, x, dtypes, shape if len(shape) == 2 else (None, None))
    return shape


def _weights(name, w, dtypes, G, N, K):
    """Expert weights [G*N, K], or the same as [G, N, K]."""
    _want(name, w, dtypes, (G, N, K) if w.dim() == 3 else (G * N, K))


def _bf16_gemm(name, a, b, offs, shape, dims, out_dtype, out, stream):
    tdt, cdt = _out_dtype(out_dtype)
    if out is None:
        out = _empty(shape, tdt, a, stream)
    else:
        _want("output", out, (tdt,), shape)
    _run(name, (a, b, offs, out), stream, a.data_ptr(), b.data_ptr(), offs.data_ptr(), *dims, out.data_ptr(), cdt)
    return out


def bf16_grouped_gemm_fwd(x, w, offs, N: int, out_dtype: str = "f32", y=None, stream=None):
    """Y [M, N] = per-expert X_g W_g^T of bf16 tensors: x [M, K], w [G*N, K] (or [G, N, K]), offs int32 [G+1].
    N % 8 == 0, K % 8 == 0."""
    bf16 = _bf16_types()
    G = _groups(offs)
    M, K = _rows("x", x, bf16)
    _weights("w", w, bf16, G, N, K)
    return _bf16_gemm("bf16_grouped_gemm_fwd", x, w, offs, (M, N), (G, M, N, K), out_dtype, y, stream)


def bf16_grouped_gemm_dgrad(dy, w, offs, K: int, out_dtype: str = "f32", dx=None, stream=None):
    """dX [M, K] = per-expert dY_g W_g of bf16 tensors: dy [M, N], w [G*N, K] (or [G, N, K]), the forward's
    weights as they are."""
    bf16 = _bf16_types()
    G = _groups(offs)
    M, N = _rows("dy", dy, bf16)
    _weights("w", w, bf16, G, N, K)
    return _bf16_gemm("bf16_grouped_gemm_dgrad", dy, w, offs, (M, K), (G, M, N, K), out_dtype, dx, stream)


def bf16_grouped_gemm_wgrad(dy, x, offs, out_dtype: str = "f32", dw=None, stream=None):
    """dW [G, N, K] = per-expert dY_g^T X_g of bf16 tensors: dy [M, N], x [M, K].  Zero for an expert without
    rows."""
    bf16 = _bf16_types()
    G = _groups(offs)
    M, N = _rows("dy", dy, bf16)
    _want("x", x, bf16, (M, None))
    K = x.shape[1]
    return _bf16_gemm("bf16_grouped_gemm_wgrad", dy, x, offs, (G, N, K), (G, M, N, K), out_dtype, dw, stream)


def _int8_rowwise(name, x, R, C, q, s, stream):
    torch = _torch()
    q = _empty((R, C), torch.int8, x, stream) if q is None else q
    s = _empty((R,), torch.float32, x, stream) if s is None else s
    _want("q", q, (torch.int8,), (R, C))
    _want("s", s, (torch.float32,), (R,))
    _run(name, (x, q, s), stream, x.data_ptr(), R, C, q.data_ptr(), s.data_ptr())
    return q, s


def int8_quantize_rowwise(x, q=None, s=None, stream=None):
    """x bf16 [R, C] -> (q int8 [R, C], s f32 [R]): s = amax / 127 of the row, q = nearest of 127 x / amax
    (tokens of activations, output channels of weights).  C % 8 == 0."""
    R, C = _rows("x", x, _bf16_types())
    return _int8_rowwise("int8_quantize_rowwise", x, R, C, q, s, stream)


def int8_quantize_swiglu_rowwise(y, q=None, s=None, stream=None):
    """y bf16 [R, 2C] (gate columns, then up columns) -> (q int8 [R, C], s f32 [R]) of silu(gate) * up."""
    R, C2 = _rows("y", y, _bf16_types())
    if C2 % 2:
        raise ValueError(f"y: expected gate and up columns, got {C2}")
    return _int8_rowwise("int8_quantize_swiglu_rowwise", y, R, C2 // 2, q, s, stream)


def int8_grouped_gemm_fwd(qx, sx, qw, sw, offs, N: int, out_dtype: str = "f32", y=None, stream=None):
    """Y [M, N] = per-expert qx_g qw_g^T (exact) times the token's and the channel's scale: qx int8 [M, K],
    sx f32 [M], qw int8 [G*N, K] (or [G, N, K]), sw f32 [G*N] (or [G, N]).  N % 8 == 0, K % 16 == 0."""
    torch = _torch()
    i8, f32 = (torch.int8,), (torch.float32,)
    G = _groups(offs)
    M, K = _rows("qx", qx, i8)
    _want("sx", sx, f32, (M,))
    _weights("qw", qw, i8, G, N, K)
    _want("sw", sw, f32, (G, N) if sw.dim() == 2 else (G * N,))
    tdt, cdt = _out_dtype(out_dtype)
    if y is None:
        y = _empty((M, N), tdt, qx, stream)
    else:
        _want("y", y, (tdt,), (M, N))
    _run("int8_grouped_gemm_fwd", (qx, sx, qw, sw, offs, y), stream, qx.data_ptr(), sx.data_ptr(), qw.data_ptr(),
         sw.data_ptr(), offs.data_ptr(), G, M, N, K, y.data_ptr(), cdt)
    return y


# ---------------------------------------------------------------- AdamW
class _AdamWTensor(ctypes.Structure):
    _fields_ = [("n", _i64)] + [(k, _p) for k in ("p", "w_bf16", "g", "m", "v", "ms", "vs")]


class _AdamWHyper(ctypes.Structure):
    _fields_ = [(k, ctypes.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
               [("step", _i64)] + [(k, _p) for k in ("lr_dev", "step_dev", "grad_scale")]


class AdamWTable:
    """The tensors of an optimizer step (adamw_table makes it): their addresses, checked once.  It keeps the
    tensors alive; make a new one when a tensor is replaced by another."""

    def __init__(self, entries, array, bits, grad_dtype, like):
        self.entries, self.array, self.bits, self.grad_dtype, self.like = entries, array, bits, grad_dtype, like
        self.args = ctypes.addressof(array), len(array), grad_dtype, bits           # (of the C call)
        self.weights = [t for row in entries for t in row[:2] if t is not None]     # (params and their copies)


def adamw_table(params, grads, exp_avg, exp_avg_sq, weights=None, exp_avg_scales=None, exp_avg_sq_scales=None):
    """Tensors of adamw_step, as lists of one length (all contiguous, on one GPU, none overlapping another that
    the step writes).

    params f32; grads all f32 or all bf16; weights (optional) the bf16 copies, entries may be None; exp_avg and
    exp_avg_sq the moments: all f32, or all uint8 with exp_avg_scales and exp_avg_sq_scales f32 [ceil(n / 128)]
    (zeros in codes and scales are zero moments)."""
    torch = _torch()
    count = len(params)
    if count == 0:
        raise ValueError("params: expected at least one tensor")
    eight = exp_avg[0].dtype == torch.uint8 if len(exp_avg) else False
    if eight != (exp_avg_scales is not None) or eight != (exp_avg_sq_scales is not None):
        raise ValueError("exp_avg_scales and exp_avg_sq_scales go with uint8 moments, and only with them")
    none = [None] * count
    lists = {"params": params, "weights": none if weights is None else weights, "grads": grads, "exp_avg": exp_avg,
             "exp_avg_sq": exp_avg_sq, "exp_avg_scales": exp_avg_scales if eight else none,
             "exp_avg_sq_scales": exp_avg_sq_scales if eight else none}
    for k, v in lists.items():
        if len(v) != count:
            raise ValueError(f"{k}: expected {count} tensors, got {len(v)}")
    gdt = grads[0].dtype
    if gdt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grads: expected float32 or bfloat16, got {gdt}")
    state = torch.uint8 if eight else torch.float32
    types = {"params": torch.float32, "weights": torch.bfloat16, "grads": gdt, "exp_avg": state, "exp_avg_sq": state,
             "exp_avg_scales": torch.float32, "exp_avg_sq_scales": torch.float32}
    array, entries, spans = (_AdamWTensor * count)(), [], []
    for i in range(count):
        row = [lists[k][i] for k in lists]
        n = params[i].numel()
        for k, t in zip(lists, row):
            if t is None:
                if k != "weights" and not (k.endswith("scales") and not eight):
                    raise ValueError(f"{k}[{i}] is None")
                continue
            want = (n + 127) // 128 if k.endswith("scales") else n
            if t.dtype != types[k]:
                raise TypeError(f"{k}[{i}]: expected {types[k]}, got {t.dtype}")
            if t.numel() != want:
                raise ValueError(f"{k}[{i}]: expected {want} elements, got {t.numel()}")
            if t.device != params[0].device:
                raise ValueError(f"{k}[{i}] is on {t.device}, params[0] on {params[0].device}")
            if want:
                spans.append((_ptr(t), _ptr(t) + want * t.element_size(), k != "grads", f"{k}[{i}]"))
        array[i] = _AdamWTensor(n, *[_ptr(t) for t in row])
        entries.append(row)
    last = None                       # of the spans so far, the one that ends last, and the last-ending written one
    wrote = None
    for s in sorted(spans):
        hit = last if s[2] else wrote
        if hit is not None and s[0] < hit[1]:
            raise ValueError(f"{s[3]} and {hit[3]} overlap")
        last = s if last is None or s[1] > last[1] else last
        if s[2]:
            wrote = s if wrote is None or s[1] > wrote[1] else wrote
    return AdamWTable(entries, array, 8 if eight else 32, MXMOE_BF16 if gdt == torch.bfloat16 else MXMOE_F32, params[0])


def adamw_step(table, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale=None, stream=None) -> None:
    """One AdamW step over the table's tensors, in place, in one launch (per 48 tensors).

    step (counted from 1) and lr are numbers, or GPU scalars (int64 / float32 tensors) that the kernel reads,
    for a step captured into a graph.  grad_scale: a float32 GPU scalar that multiplies every gradient
    (clipping), or None.

    The weights and their copies count as modified in place, so a backward pass that saved one before the step
    raises; replays of a captured step cannot be noticed that way."""
    torch = _torch()
    hyper = _AdamWHyper(0.0, beta1, beta2, eps, weight_decay, 1)
    scalars = []
    if isinstance(lr, torch.Tensor):
        scalars.append(("lr", lr, torch.float32, "lr_dev"))
    else:
        hyper.lr = lr
    if isinstance(step, torch.Tensor):
        scalars.append(("step", step, torch.int64, "step_dev"))
    else:
        hyper.step = int(step)
    if grad_scale is not None:
        scalars.append(("grad_scale", grad_scale, torch.float32, "grad_scale"))
    for name, t, dt, field in scalars:
        if t.dtype != dt or t.numel() != 1:
            raise TypeError(f"{name}: expected one {dt} on the GPU, got {t.dtype} of {t.numel()}")
        setattr(hyper, field, _ptr(t))
    _run("adamw_step", (table.like, *[t for _, t, _, _ in scalars]) if scalars else (table.like,), stream, *table.args,
         ctypes.addressof(hyper))
    torch.autograd.graph.increment_version(table.weights)


def adamw_dequantize(q, s, moment: str, out_dtype: str = "f32", out=None, stream=None):
    """Values of 8-bit moments: q uint8 (any shape), s f32 [ceil(n / 128)], moment "exp_avg" or "exp_avg_sq"
    (their codes differ); out has q's shape."""
    torch = _torch()
    if moment not in ("exp_avg", "exp_avg_sq"):
        raise ValueError(f"moment: expected 'exp_avg' or 'exp_avg_sq', got {moment!r}")
    _want("q", q, (torch.uint8,), q.shape)
    _want("s", s, (torch.float32,), ((q.numel() + 127) // 128,))
    tdt, cdt = _out_dtype(out_dtype)
    if out is None:
        out = _empty(q.shape, tdt, q, stream)
    else:
        _want("out", out, (tdt,), q.shape)
    _run("adamw_dequantize", (q, s, out), stream, q.data_ptr(), s.data_ptr(), q.numel(), int(moment == "exp_avg_sq"),
         out.data_ptr(), cdt)
    return out


# ---------------------------------------------------------------- norm
@functools.lru_cache(None)
def _floats():
    """The element types of the norm's and the rows' tensors, and their codes."""
    torch = _torch()
    return {torch.float32: MXMOE_F32, torch.bfloat16: MXMOE_BF16}


def _norm_inputs(x, w, residual, h, stream):
    """Checked arguments of a norm: the tensors, the C call's first arguments, its h."""
    floats = _floats()
    R, C = _rows("x", x, floats)
    _want("w", w, floats, (C,))
    if residual is None:
        if h is not None:
            raise ValueError("h goes with residual, and only with it")
        return (x, w), (x.data_ptr(), floats[x.dtype], None, 0, w.data_ptr(), floats[w.dtype], R, C), None
    _want("residual", residual, floats, (R, C))
    h = _out(h, "h", (R, C), residual.dtype, x, stream)
    return (x, w, residual, h), (x.data_ptr(), floats[x.dtype], residual.data_ptr(), floats[residual.dtype],
                                 w.data_ptr(), floats[w.dtype], R, C), h


def rmsnorm_fwd(x, w, eps: float = 1e-6, residual=None, out_dtype: str = "bf16", y=None, h=None, stream=None):
    """Root-mean-square norm y [R, C] = h / sqrt(mean(h^2) + eps) * w of x [R, C], and with residual [R, C] of
    h = x + residual rounded to the residual's type, which is returned too: y, or (y, h).

    x, residual and w [C] are f32 or bf16 each.  h may be the residual itself (updated in place).  C % 8 == 0,
    C <= 32768."""
    tensors, args, h = _norm_inputs(x, w, residual, h, stream)
    tdt, cdt = _out_dtype(out_dtype)
    y = _out(y, "y", x.shape, tdt, x, stream)
    _run("rmsnorm_fwd", (*tensors, y), stream, *args, eps, y.data_ptr(), cdt, None if h is None else h.data_ptr())
    return y if h is None else (y, h)


def _quantize_rmsnorm(name, x, w, eps, residual, with_y, q, s, h, y, stream, qdt, sdt, sshape):
    tensors, args, h = _norm_inputs(x, w, residual, h, stream)
    q = _out(q, "q", x.shape, qdt, x, stream)
    s = _out(s, "s", sshape, sdt, x, stream)
    tensors += (q, s)
    if y is not None or with_y:
        y = _out(y, "y", x.shape, _torch().bfloat16, x, stream)
        tensors += (y,)
    _run(name, tensors, stream, *args, eps, q.data_ptr(), s.data_ptr(), None if y is None else y.data_ptr(),
         None if h is None else h.data_ptr())
    return (q, s) + (() if h is None else (h,)) + (() if y is None else (y,))


def int8_quantize_rmsnorm_rowwise(x, w, eps: float = 1e-6, residual=None, with_y: bool = False, q=None, s=None, h=None,
                                  y=None, stream=None):
    """rmsnorm_fwd's y as 8-bit integers with a scale per row (as int8_quantize_rowwise's, in one rounding from the
    exact values): (q int8 [R, C], s f32 [R]), then h with a residual, then y in bf16 with `with_y`."""
    torch = _torch()
    return _quantize_rmsnorm("int8_quantize_rmsnorm_rowwise", x, w, eps, residual, with_y, q, s, h, y, stream, torch.int8,
                             torch.float32, x.shape[:1])


def mx_quantize_rmsnorm_rowwise(x, w, eps: float = 1e-6, residual=None, with_y: bool = False, q=None, s=None, h=None,
                                y=None, stream=None):
    """rmsnorm_fwd's y as E4M3 codes with a scale per 32 (as mx_quantize_rowwise's, in one rounding from the exact
    values): (q uint8 [R, C], s uint8 [R, C/32]), then h with a residual, then y in bf16 with `with_y`."""
    u8 = _torch().uint8
    return _quantize_rmsnorm("mx_quantize_rmsnorm_rowwise", x, w, eps, residual, with_y, q, s, h, y, stream, u8, u8,
                             (*x.shape[:1], x.shape[-1] // 32))


def rmsnorm_bwd(dy, h, w, eps: float = 1e-6, dres=None, dx=None, dw=None, need_dw: bool = True, stream=None):
    """Gradients of rmsnorm_fwd's y with respect to h [R, C] (which is that of x and of the residual) and w:
    (dx of h's type [R, C], dw f32 [C], or None without need_dw).

    dy [R, C] f32 or bf16; dres, of h's type, is the gradient that reaches h by another way and is added (dx may be dres
    itself)."""
    torch = _torch()
    floats = _floats()
    R, C = _rows("h", h, floats)
    _want("dy", dy, floats, (R, C))
    _want("w", w, floats, (C,))
    tensors = (dy, h, w)
    if dres is not None:
        _want("dres", dres, (h.dtype,), (R, C))
        tensors += (dres,)
    dx = _out(dx, "dx", (R, C), h.dtype, h, stream)
    tensors += (dx,)
    ws = None
    if need_dw:
        dw = _out(dw, "dw", (C,), torch.float32, h, stream)
        ws = _out(None, "ws", (max(0, lib().rmsnorm_bwd_workspace(R, C)),), torch.uint8, h, stream)
        tensors += (dw,)
    elif dw is not None:
        raise ValueError("dw goes with need_dw")
    _run("rmsnorm_bwd", tensors, stream, dy.data_ptr(), floats[dy.dtype], h.data_ptr(), floats[h.dtype], w.data_ptr(),
         floats[w.dtype], None if dres is None else dres.data_ptr(), R, C, eps, dx.data_ptr(),
         None if dw is None else dw.data_ptr(), None if ws is None else ws.data_ptr())
    return dx, dw


# ---------------------------------------------------------------- routing
_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score: expected 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def _route(name, logits, top, score, bias, groups, keep_groups, group_top, renormalize, scale, valid, ids, weights, sort,
           stream):
    torch = _torch()
    floats = _floats()
    T, E = _rows("logits", logits, floats)
    tensors = (logits,)
    if bias is not None:
        _want("bias", bias, (torch.float32,), (E,))
        tensors += (bias,)
    if valid is not None:
        _want("valid", valid, (torch.bool, torch.uint8), (T,))
        tensors += (valid,)
    ids = _out(ids, "ids", (T, top), torch.int32, logits, stream)
    weights = _out(weights, "weights", (T, top), torch.float32, logits, stream)
    _run(name, (*tensors, ids, weights, *sort[0]), stream, logits.data_ptr(), floats[logits.dtype],
         None if bias is None else bias.data_ptr(), None if valid is None else valid.data_ptr(), T, E, top, _score(score),
         groups, groups if keep_groups is None else keep_groups, group_top, int(renormalize), scale, ids.data_ptr(),
         weights.data_ptr(), *sort[1])
    return ids, weights


def moe_route_fwd(logits, top: int, score: str = "softmax", bias=None, groups: int = 1, keep_groups: Optional[int] = None,
                  group_top: int = 1, renormalize: bool = True, scale: float = 1.0, valid=None, ids=None, weights=None,
                  stream=None):
    """The `top` experts of each token and their weights from router logits [T, E] (f32 or bf16): (ids int32 [T, top],
    weights f32 [T, top]).

    The choice goes by c: the softmax or sigmoid scores plus bias f32 [E] (which balances and does not weigh), or without
    a bias the logits, which order the experts alike.  Of `groups` groups of consecutive experts only the keep_groups with
    the largest sum of their group_top (1 or 2) best c stay: with group_top=2 and no bias these are sums of two logits, which
    do not order the groups as sums of scores do (a bias of zeros gives those).  Equal ones: the lower index.  Weights are
    the scores, divided by their sum if renormalize, times scale.  valid (bool [T]): tokens that are False get ids of -1 and
    weights of 0.  A bias of -infinity keeps an expert out of every choice in which enough others are left; large finite
    biases do so too and are slower, since scores are resolved relative to the largest |c|."""
    return _route("moe_route_fwd", logits, top, score, bias, groups, keep_groups, group_top, renormalize, scale, valid,
                  ids, weights, ((), ()), stream)


def _sort_outputs(T, top, G, first, offs, row_idx, pos, like, stream):
    i32 = _torch().int32
    offs = _out(offs, "offs", (G + 1,), i32, like, stream)
    row_idx = _out(row_idx, "row_idx", (T * top,), i32, like, stream)
    pos = _out(pos, "pos", (T, top), i32, like, stream)
    need = lib().moe_sort_workspace(T * top, G)
    ws = _out(None, "ws", (need,), _torch().uint8, like, stream) if need > 0 else None
    return (offs, row_idx, pos), (G, first, offs.data_ptr(), row_idx.data_ptr(), pos.data_ptr(),
                                  None if ws is None else ws.data_ptr()), ws


def moe_sort(ids, G: int, first: int = 0, offs=None, row_idx=None, pos=None, stream=None):
    """The chosen pairs ids int32 [T, top] by expert, for the G experts from `first` on that are here: (offs int32
    [G+1], row_idx int32 [T*top] the token of each row, pos int32 [T, top] the row of each pair).

    An expert's rows keep the order of their tokens.  Pairs of other experts and negative ids have no row: pos -1, and
    row_idx is -1 from offs[G] on."""
    T, top = _rows("ids", ids, (_torch().int32,))
    out, args, ws = _sort_outputs(T, top, G, first, offs, row_idx, pos, ids, stream)
    _run("moe_sort", (ids, *out), stream, ids.data_ptr(), T, top, *args)
    return out


def moe_route_sort(logits, top: int, G: Optional[int] = None, first: int = 0, score: str = "softmax", bias=None,
                   groups: int = 1, keep_groups: Optional[int] = None, group_top: int = 1, renormalize: bool = True,
                   scale: float = 1.0, valid=None, ids=None, weights=None, offs=None, row_idx=None, pos=None, stream=None):
    """moe_route_fwd and moe_sort at once: (ids, weights, offs, row_idx, pos).  G: the experts here (all)."""
    T, E = _rows("logits", logits, _floats())
    out, args, ws = _sort_outputs(T, top, E if G is None else G, first, offs, row_idx, pos, logits, stream)
    return (*_route("moe_route_sort", logits, top, score, bias, groups, keep_groups, group_top, renormalize, scale, valid,
                    ids, weights, (out, args), stream), *out)


def moe_route_bwd(dweights, ids, logits, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                  dlogits=None, stream=None):
    """dlogits [T, E] (of the logits' type) from dweights f32 [T, top], with the forward call's ids and logits."""
    torch = _torch()
    floats = _floats()
    T, E = _rows("logits", logits, floats)
    _want("ids", ids, (torch.int32,), (T, None))
    _want("dweights", dweights, (torch.float32,), ids.shape)
    dlogits = _out(dlogits, "dlogits", (T, E), logits.dtype, logits, stream)
    _run("moe_route_bwd", (dweights, ids, logits, dlogits), stream, dweights.data_ptr(), ids.data_ptr(), logits.data_ptr(),
         floats[logits.dtype], T, E, ids.shape[1], _score(score), int(renormalize), scale, dlogits.data_ptr())
    return dlogits


# ---------------------------------------------------------------- rows out and back
def _pairs(pos, weights, T):
    """Checked pos [T, top] and weights of the rows' entry points: top."""
    torch = _torch()
    _want("pos", pos, (torch.int32,), (T, None))
    if weights is not None:
        _want("weights", weights, (torch.float32,), pos.shape)
    return pos.shape[1]


def moe_dispatch(x, pos, scales=None, rows: Optional[int] = None, xr=None, sr=None, stream=None):
    """Tokens' rows to their experts' places: xr[pos[t, k]] = x[t] for x [T, C] (bf16, f32, int8 or uint8) and pos int32
    [T, top] (moe_sort's): xr [rows, C], rows T * top unless given.  With scales [T] or [T, S] of the rows (f32 or uint8)
    also sr[pos[t, k]] = scales[t]: (xr, sr).  Rows that no pair names stay as they were."""
    torch = _torch()
    T, C = _rows("x", x, (torch.bfloat16, torch.float32, torch.int8, torch.uint8))
    top = _pairs(pos, None, T)
    M = (T * top if rows is None else rows) if xr is None else xr.shape[0]
    xr = _out(xr, "xr", (M, C), x.dtype, x, stream)
    if scales is None:
        if sr is not None:
            raise ValueError("sr goes with scales")
        _run("moe_dispatch", (x, pos, xr), stream, x.data_ptr(), C * x.element_size(), None, 0, pos.data_ptr(), T, top, M,
             xr.data_ptr(), None)
        return xr
    shape = scales.shape[1:]
    _want("scales", scales, (torch.float32, torch.uint8), (T, *shape))
    sr = _out(sr, "sr", (M, *shape), scales.dtype, x, stream)
    _run("moe_dispatch", (x, pos, scales, xr, sr), stream, x.data_ptr(), C * x.element_size(), scales.data_ptr(),
         shape.numel() * scales.element_size(), pos.data_ptr(), T, top, M, xr.data_ptr(), sr.data_ptr())
    return xr, sr


def moe_combine_fwd(y, pos, weights=None, residual=None, out_dtype: str = "bf16", out=None, stream=None):
    """Weighted sums of the tokens' rows: out [T, C] = residual + sum_k weights[t, k] y[pos[t, k]] for y [M, C], pos int32
    [T, top] (moe_sort's; pairs without a row add nothing), weights f32 [T, top] (None: 1, which is moe_dispatch's
    backward) and residual [T, C] (None: 0).  y and residual are f32 or bf16 each; out may be the residual itself."""
    floats = _floats()
    M, C = _rows("y", y, floats)
    T = pos.shape[0]
    top = _pairs(pos, weights, T)
    tdt, cdt = _out_dtype(out_dtype)
    tensors = (y, pos)
    if weights is not None:
        tensors += (weights,)
    if residual is not None:
        _want("residual", residual, floats, (T, C))
        tensors += (residual,)
    out = _out(out, "out", (T, C), tdt, y, stream)
    _run("moe_combine_fwd", (*tensors, out), stream, y.data_ptr(), floats[y.dtype], pos.data_ptr(),
         None if weights is None else weights.data_ptr(), None if residual is None else residual.data_ptr(),
         0 if residual is None else floats[residual.dtype], T, top, M, C, out.data_ptr(), cdt)
    return out


def moe_combine_bwd(dout, pos, weights=None, y=None, out_dtype: Optional[str] = None, rows: Optional[int] = None, dy=None,
                    need_dy: bool = True, stream=None):
    """Gradients of moe_combine_fwd's out [T, C] with respect to y and the weights: (dy [M, C] with dy[pos[t, k]] =
    weights[t, k] dout[t], dweights f32 [T, top] with the products of dout[t] and y[pos[t, k]], 0 for a pair
    without a row).

    y [M, C]: the forward call's (without it dweights is None, and dy has `rows` rows, T * top unless given, of
    out_dtype).  dy is of y's type and may be y itself; rows of it that no pair names stay as they were; it is None
    without need_dy.  The residual's gradient is dout."""
    torch = _torch()
    floats = _floats()
    T, C = _rows("dout", dout, floats)
    top = _pairs(pos, weights, T)
    tensors = (dout, pos)
    if weights is not None:
        tensors += (weights,)
    dweights = None
    if y is not None:
        _want("y", y, floats, (None, C))
        M, dt = y.shape[0], y.dtype
        if out_dtype is not None and _out_dtype(out_dtype)[0] != dt:
            raise TypeError(f"out_dtype: dy is of y's type, {dt}")
        dweights = _out(None, "dweights", (T, top), torch.float32, dout, stream)
        tensors += (y, dweights)
    else:
        M = (T * top if rows is None else rows) if dy is None else dy.shape[0]
        dt = _out_dtype("bf16" if out_dtype is None else out_dtype)[0] if dy is None or out_dtype is not None else dy.dtype
    if need_dy:
        if dt not in floats:
            raise TypeError(f"dy: expected float32 or bfloat16, got {dt}")
        dy = _out(dy, "dy", (M, C), dt, dout, stream)
        tensors += (dy,)
    elif dy is not None:
        raise ValueError("dy goes with need_dy")
    _run("moe_combine_bwd", tensors, stream, dout.data_ptr(), floats[dout.dtype], pos.data_ptr(),
         None if weights is None else weights.data_ptr(), None if y is None else y.data_ptr(), floats[dt], T, top, M, C,
         None if dy is None else dy.data_ptr(), None if dweights is None else dweights.data_ptr())
    return dy, dweights
