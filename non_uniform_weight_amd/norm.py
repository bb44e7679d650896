"""The root-mean-square norm in front of a decoder's products, with the residual's addition (include/sqllm_norm.h).

The output is fp16, or already in the stored form that int8_gemm and int8_glu (rms_norm_int8) or fp8_gemm
(rms_norm_fp8) take as x and x_scale."""
from __future__ import annotations

import ctypes

import torch

from . import _calls, _check, _lib
from .fp8 import fp8_cols, fp8_scale_pitch
from .int8 import int8_cols

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_row = [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _f32, _vp]
_lib.sqllm_rms_norm.restype = _i32
_lib.sqllm_rms_norm.argtypes = [*_row, _vp, _vp]
for _f in (_lib.sqllm_rms_norm_int8, _lib.sqllm_rms_norm_fp8):
    _f.restype = _i32
    _f.argtypes = [*_row, _vp, _vp, _vp]

EXPORTS = ("sqllm_rms_norm", "sqllm_rms_norm_int8", "sqllm_rms_norm_fp8")
_half, _int8, _fp8 = _lib.sqllm_rms_norm, _lib.sqllm_rms_norm_int8, _lib.sqllm_rms_norm_fp8


def _half_output(t, name, x, rows, cols, index):
    """As _calls.output, for one that is like x."""
    if t is None and x.is_contiguous():  # half a microsecond less than by shape, type and device
        t = torch.empty_like(x)
        return t, t.data_ptr()
    return _calls.output(t, name, (rows, cols), torch.float16, index)


def _inputs(x, weight, eps, residual, total, index):
    """(rows, cols, the C calls' arguments up to sum, sum); sum as a tuple of none or one."""
    rows, cols, ldx, xp = _calls.half_rows(x, "x", index)
    wp = _calls.address(weight, "weight", torch.float16, index)
    if weight.shape != (cols,):
        raise ValueError(f"weight: shape {(cols,)} expected, got {tuple(weight.shape)}")
    if residual is None:
        if total is not None:
            raise ValueError("total: only with a residual")
        return rows, cols, (xp, ldx, None, 0, wp, rows, cols, eps, None), ()
    added, width, ldr, rp = _calls.half_rows(residual, "residual", index)
    if added != rows or width != cols:
        raise ValueError(f"residual: shape {(rows, cols)} expected, got {(added, width)}")
    total, tp = _half_output(total, "total", x, rows, cols, index)
    return rows, cols, (xp, ldx, rp, ldr, wp, rows, cols, eps, tp), (total,)


@_calls.on_stream
def rms_norm(index, handle, x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
             y: torch.Tensor | None = None, total: torch.Tensor | None = None):
    """y [rows, cols] = x / sqrt(mean(x^2) + eps) * weight for fp16 x [rows, cols] and weight [cols]; with a residual
    (y, total): the norm of total = x + residual.  total may be x or residual itself; the rows of x and residual may
    be further apart than cols.  stream: as for every call (keyword)."""
    rows, cols, args, total = _inputs(x, weight, eps, residual, total, index)
    y, yp = _half_output(y, "y", x, rows, cols, index)
    _check(_half(*args, yp, handle), "sqllm_rms_norm")
    return (y, *total) if total else y


@_calls.on_stream
def rms_norm_int8(index, handle, x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                  q: torch.Tensor | None = None, scale: torch.Tensor | None = None, total: torch.Tensor | None = None):
    """(q, scale), with a residual (q, scale, total): rms_norm, its y in the form of int8_quantize."""
    rows, cols, args, total = _inputs(x, weight, eps, residual, total, index)
    q, qp = _calls.output(q, "q", (rows, int8_cols(cols)), torch.int8, index)
    scale, sp = _calls.output(scale, "scale", (rows,), torch.float32, index)
    _check(_int8(*args, qp, sp, handle), "sqllm_rms_norm_int8")
    return q, scale, *total


@_calls.on_stream
def rms_norm_fp8(index, handle, x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                 q: torch.Tensor | None = None, scale: torch.Tensor | None = None, total: torch.Tensor | None = None):
    """(q, scale), with a residual (q, scale, total): rms_norm, its y in the form of fp8_quantize."""
    rows, cols, args, total = _inputs(x, weight, eps, residual, total, index)
    q, qp = _calls.output(q, "q", (rows, fp8_cols(cols)), torch.uint8, index)
    scale, sp = _calls.output(scale, "scale", (rows, fp8_scale_pitch(cols)), torch.uint8, index)
    _check(_fp8(*args, qp, sp, handle), "sqllm_rms_norm_fp8")
    return q, scale, *total
