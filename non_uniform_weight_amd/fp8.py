"""Block-scaled 8-bit floating point weights: the quantiser and the product (include/sqllm_fp8.h).

A matrix is stored as e4m3 codes, uint8 [rows, fp8_cols(cols)], and power-of-two scales, one byte (exponent + 127)
for each row and block of 128 columns, uint8 [rows, fp8_scale_pitch(cols)].  The product rounds its fp16
activations to the same form and runs on the matrix cores, at any batch."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _calls, _check, _lib

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_lib.sqllm_fp8_cols.restype = _i64
_lib.sqllm_fp8_cols.argtypes = [_i64]
_lib.sqllm_fp8_scale_pitch.restype = _i64
_lib.sqllm_fp8_scale_pitch.argtypes = [_i64]
_lib.sqllm_fp8_quantize.restype = _i32
_lib.sqllm_fp8_quantize.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
for _size in (_lib.sqllm_fp8_workspace_bytes, _lib.sqllm_fp8_stored_workspace_bytes):
    _size.restype = _sz
    _size.argtypes = [_i64, _i64, _i64]
_lib.sqllm_fp8_gemm.restype = _i32
_lib.sqllm_fp8_gemm.argtypes = [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp]
_lib.sqllm_fp8_gemm_stored.restype = _i32
_lib.sqllm_fp8_gemm_stored.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _sz, _vp]

EXPORTS = ("sqllm_fp8_cols", "sqllm_fp8_scale_pitch", "sqllm_fp8_quantize", "sqllm_fp8_workspace_bytes",
           "sqllm_fp8_stored_workspace_bytes", "sqllm_fp8_gemm", "sqllm_fp8_gemm_stored")
_gemm, _gemm_stored = _lib.sqllm_fp8_gemm, _lib.sqllm_fp8_gemm_stored


@functools.lru_cache(maxsize=4096)
def fp8_cols(cols: int) -> int:
    """Columns of the stored codes: cols rounded up to 128 (0 if out of range)."""
    return int(_lib.sqllm_fp8_cols(cols)) if _calls.held(_i64, cols) else 0


@functools.lru_cache(maxsize=4096)
def fp8_scale_pitch(cols: int) -> int:
    """Bytes of a row of scales: one per block of 128 columns, rounded up to 4 (0 if out of range)."""
    return int(_lib.sqllm_fp8_scale_pitch(cols)) if _calls.held(_i64, cols) else 0


@functools.lru_cache(maxsize=4096)
def fp8_workspace_bytes(rows: int, cols: int, batch: int, stored: bool = False) -> int:
    """Scratch bytes of fp8_gemm for x in fp16, or (stored) in e4m3 with x_scale: far less."""
    size = _lib.sqllm_fp8_stored_workspace_bytes if stored else _lib.sqllm_fp8_workspace_bytes
    return int(size(rows, cols, batch)) if _calls.held(_i64, rows, cols, batch) else 0


@_calls.on_stream
def fp8_quantize(index, handle, x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """(q, scale) of fp16 x [rows, cols]; the columns of a row are adjacent, rows may be further apart than cols.
    Offline for weights; the product rounds its activations itself.  stream: as for every call (keyword)."""
    if x.dim() != 2 or x.numel() == 0:
        raise ValueError(f"x: shape (rows, cols) expected, got {tuple(x.shape)}")
    if x.dtype is not torch.float16:
        raise TypeError(f"x: dtype torch.float16 expected, got {x.dtype}")
    rows, cols = x.shape
    if cols > 1 and x.stride(1) != 1:
        raise ValueError("x: adjacent columns expected")
    q, qp = _calls.output(q, "q", (rows, fp8_cols(cols)), torch.uint8, index)
    scale, sp = _calls.output(scale, "scale", (rows, fp8_scale_pitch(cols)), torch.uint8, index)
    _check(_lib.sqllm_fp8_quantize(x.data_ptr(), rows, cols, x.stride(0) if rows > 1 else cols, qp, sp, handle),
           "sqllm_fp8_quantize")
    return q, scale


@_calls.on_stream
def fp8_gemm(index, handle, q: torch.Tensor, scale: torch.Tensor, x: torch.Tensor, y: torch.Tensor | None = None,
             ws: torch.Tensor | None = None, *, x_scale: torch.Tensor | None = None) -> torch.Tensor:
    """y [batch, rows] = x W^T for fp16 x [batch, cols] (or [cols]) and W stored as fp8_quantize leaves it; with
    x_scale, x and x_scale are in that form too (as rms_norm_fp8 leaves them).
    ws: scratch of fp8_workspace_bytes(rows, cols, batch, stored=x_scale is not None) bytes (a cached one if None)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x: torch.Tensor expected")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2 or q.dim() != 2:
        raise ValueError(f"x: shape (batch, cols), q: shape (rows, columns) expected, got {tuple(x.shape)}, "
                         f"{tuple(q.shape)}")
    batch, cols = x.shape
    rows, kept = q.shape
    pitch = fp8_scale_pitch(cols)
    if kept != (cols if x_scale is not None else fp8_cols(cols)) or scale.shape != (rows, pitch):
        raise ValueError(f"q, scale: shapes {(rows, fp8_cols(cols))} and {(rows, pitch)} expected for "
                         f"{cols} columns, got {tuple(q.shape)} and {tuple(scale.shape)}")
    qp, sp = _calls.address(q, "q", torch.uint8, index), _calls.address(scale, "scale", torch.uint8, index)
    if x_scale is not None:
        call, name = _gemm_stored, "sqllm_fp8_gemm_stored"
        xs = (_calls.address(x, "x", torch.uint8, index), _calls.address(x_scale, "x_scale", torch.uint8, index))
        if cols != fp8_cols(cols) or x_scale.shape != (batch, pitch):
            raise ValueError(f"x, x_scale: shapes {(batch, fp8_cols(cols))} and {(batch, pitch)} expected, got "
                             f"{tuple(x.shape)} and {tuple(x_scale.shape)}")
    else:
        call, name, xs = _gemm, "sqllm_fp8_gemm", (_calls.address(x, "x", torch.float16, index),)
    y, yp = _calls.output(y, "y", (batch, rows), torch.float16, index)
    _check(_calls.with_scratch(ws, fp8_workspace_bytes(rows, cols, batch, x_scale is not None), index, handle, call, qp, sp,
                               rows, cols, *xs, batch, yp), name)
    return y
