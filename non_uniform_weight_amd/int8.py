"""Products in 8-bit integers with a scale for each token and channel (include/sqllm_int8.h).

A matrix is stored as integers, int8 [rows, int8_cols(cols)] with zeros behind the columns, and one fp32 scale for
each row.  Activations come in the same form, as int8_quantize and rms_norm_int8 leave them, or in fp16."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _calls, _check, _lib

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_lib.sqllm_int8_cols.restype = _i64
_lib.sqllm_int8_cols.argtypes = [_i64]
_lib.sqllm_int8_quantize.restype = _i32
_lib.sqllm_int8_quantize.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
for _size in (_lib.sqllm_int8_workspace_bytes, _lib.sqllm_int8_glu_workspace_bytes,
              _lib.sqllm_int8_stored_workspace_bytes, _lib.sqllm_int8_glu_stored_workspace_bytes):
    _size.restype = _sz
    _size.argtypes = [_i64, _i64, _i64]
_lib.sqllm_int8_gemm.restype = _i32
_lib.sqllm_int8_gemm.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _sz, _vp]
_lib.sqllm_int8_glu.restype = _i32
_lib.sqllm_int8_glu.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _sz, _vp]
_lib.sqllm_test_int8_plan.restype = _i32
_lib.sqllm_test_int8_plan.argtypes = [_i64, _i64, _i64, _i32, _i32, ctypes.POINTER(_i32)]

EXPORTS = ("sqllm_int8_cols", "sqllm_int8_quantize", "sqllm_int8_workspace_bytes", "sqllm_int8_glu_workspace_bytes",
           "sqllm_int8_stored_workspace_bytes", "sqllm_int8_glu_stored_workspace_bytes", "sqllm_int8_gemm",
           "sqllm_int8_glu", "sqllm_test_int8_plan")
_MAX_COLS = 131071
_gemm, _glu, _quantize = _lib.sqllm_int8_gemm, _lib.sqllm_int8_glu, _lib.sqllm_int8_quantize


@functools.lru_cache(maxsize=4096)
def int8_cols(cols: int) -> int:
    """Columns of the stored integers: cols rounded up to 128 (0 if out of range)."""
    return int(_lib.sqllm_int8_cols(cols)) if _calls.held(_i64, cols) else 0


@functools.lru_cache(maxsize=4096)
def int8_workspace_bytes(rows: int, cols: int, batch: int, stored: bool = False) -> int:
    """Scratch bytes of int8_gemm for x in fp16, or (stored) in integers with x_scale: far less."""
    size = _lib.sqllm_int8_stored_workspace_bytes if stored else _lib.sqllm_int8_workspace_bytes
    return int(size(rows, cols, batch)) if _calls.held(_i64, rows, cols, batch) else 0


@functools.lru_cache(maxsize=4096)
def int8_glu_workspace_bytes(rows: int, cols: int, batch: int, stored: bool = False) -> int:
    """The same of int8_glu."""
    size = _lib.sqllm_int8_glu_stored_workspace_bytes if stored else _lib.sqllm_int8_glu_workspace_bytes
    return int(size(rows, cols, batch)) if _calls.held(_i64, rows, cols, batch) else 0


@_calls.on_stream
def int8_quantize(index, handle, x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """(q, scale) of fp16 x [rows, cols]; the columns of a row are adjacent, rows may be further apart than cols.
    Offline for weights; for activations that several products take.  stream: as for every call (keyword)."""
    rows, cols, ldx, xp = _calls.half_rows(x, "x", index)
    q, qp = _calls.output(q, "q", (rows, int8_cols(cols)), torch.int8, index)
    scale, sp = _calls.output(scale, "scale", (rows,), torch.float32, index)
    _check(_quantize(xp, rows, cols, ldx, qp, sp, handle), "sqllm_int8_quantize")
    return q, scale


def _activations(x, x_scale, kept, index):
    """(batch, columns, address, address of the scales) of a product's x; kept: columns of the stored weights."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x: torch.Tensor expected")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2:
        raise ValueError(f"x: shape (batch, cols) expected, got {tuple(x.shape)}")
    batch, cols = x.shape
    if x_scale is None:
        if kept != int8_cols(cols):
            raise ValueError(f"weights: {int8_cols(cols)} stored columns expected for {cols} of x, got {kept}")
        return batch, cols, _calls.address(x, "x", torch.float16, index), None
    xp, xsp = _calls.address(x, "x", torch.int8, index), _calls.address(x_scale, "x_scale", torch.float32, index)
    stored, cols = cols, min(cols, _MAX_COLS)  # (the longest rows' last stored column is padding)
    if stored != kept or kept != int8_cols(cols):
        raise ValueError(f"x: the weights' {kept} stored columns (a multiple of 128) expected, got {stored}")
    if x_scale.numel() != batch:
        raise ValueError(f"x_scale: {batch} values expected, got {x_scale.numel()}")
    return batch, cols, xp, xsp


def _weights(q, scale, name, index):
    qp, sp = _calls.address(q, name, torch.int8, index), _calls.address(scale, f"{name}'s scale", torch.float32, index)
    if q.dim() != 2 or scale.shape != q.shape[:1]:
        raise ValueError(f"{name}: shapes (rows, columns) and (rows,) expected, got {tuple(q.shape)}, {tuple(scale.shape)}")
    return qp, sp


@_calls.on_stream
def int8_gemm(index, handle, q: torch.Tensor, scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor | None = None,
              y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """y fp16 [batch, rows] = x W^T for W stored as int8_quantize leaves it.  x: fp16 [batch, cols] (or [cols]),
    rounded inside; or, with x_scale (fp32 [batch]), int8 [batch, int8_cols(cols)].
    ws: scratch of int8_workspace_bytes(rows, cols, batch, stored=x_scale is not None) bytes (a cached one if None)."""
    qp, sp = _weights(q, scale, "q", index)
    rows, kept = q.shape
    batch, cols, xp, xsp = _activations(x, x_scale, kept, index)
    y, yp = _calls.output(y, "y", (batch, rows), torch.float16, index)
    _check(_calls.with_scratch(ws, int8_workspace_bytes(rows, cols, batch, xsp is not None), index, handle, _gemm, qp, sp,
                               rows, cols, xp, xsp, batch, yp), "sqllm_int8_gemm")
    return y


@_calls.on_stream
def int8_glu(index, handle, gate: torch.Tensor, gate_scale: torch.Tensor, up: torch.Tensor, up_scale: torch.Tensor,
             x: torch.Tensor, x_scale: torch.Tensor | None = None, h: torch.Tensor | None = None,
             ws: torch.Tensor | None = None) -> torch.Tensor:
    """h fp16 [batch, rows] = silu(x G^T) * (x U^T): both projections of a gated feed-forward block, the activation
    and the product in one call.  gate, up: as int8_quantize leaves them; x, x_scale: as int8_gemm's.
    ws: scratch of int8_glu_workspace_bytes(rows, cols, batch, stored=x_scale is not None) bytes (a cached one if
    None)."""
    gp, gsp = _weights(gate, gate_scale, "gate", index)
    up_, usp = _weights(up, up_scale, "up", index)
    if gate.shape != up.shape:
        raise ValueError(f"gate, up: the same shape expected, got {tuple(gate.shape)}, {tuple(up.shape)}")
    rows, kept = gate.shape
    batch, cols, xp, xsp = _activations(x, x_scale, kept, index)
    h, hp = _calls.output(h, "h", (batch, rows), torch.float16, index)
    _check(_calls.with_scratch(ws, int8_glu_workspace_bytes(rows, cols, batch, xsp is not None), index, handle, _glu, gp,
                               gsp, up_, usp, rows, cols, xp, xsp, batch, hp), "sqllm_int8_glu")
    return h


TILES = ("256x256", "256x128", "128x128", "128x64", "64x64", "64x32", "32x16", "32x16 in four groups", "32x32", "32x64",
         "64x64 in three groups")


def int8_plan(rows: int, cols: int, batch: int, gated: bool = False, stored: bool = False) -> dict:
    """Test-only: how int8_gemm (gated: int8_glu) would compute a product, without a device.  rounded_first: whether
    the quantiser's launch comes before; form: "vector" (with the rows of x the kernel holds and the chunks a wave
    has), "matrix" (with the blocks a wave has) or "tiles" (with the tile, the splits of the columns and the whole
    tiles in front of halves, 0 without)."""
    out = (_i32 * 5)()
    _check(_lib.sqllm_test_int8_plan(rows, cols, batch, gated, stored, out), "sqllm_test_int8_plan")
    plan = {"rounded_first": bool(out[0]), "form": ("vector", "matrix", "tiles")[out[1]]}
    if out[1] == 0:
        return {**plan, "held": out[2], "chunks": out[3]}
    if out[1] == 1:
        return {**plan, "blocks": out[2]}
    return {**plan, "tile": TILES[out[2]], "splits": out[3], "whole": out[4]}
