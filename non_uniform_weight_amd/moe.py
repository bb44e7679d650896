"""A mixture-of-experts layer for up to 16 tokens whose experts are dense-and-sparse LUT matrices
(include/sqllm_moe.h): the router's choice, the experts' products, and both as one call.

A projection of the experts is a dict like a group product's item, over all experts: packed (the experts' packed
matrices one after another), lut (fp16 [experts, rows, 2^bits]) and, with outliers, one CSR over the experts' rows:
row_ptr (int32 [experts * rows + 1]), col (uint16 or int16 bits), val (fp16)."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _calls, _check, _lib, packed_bytes

_vp, _i64, _i32, _sz, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


class Experts(ctypes.Structure):
    """One projection of every expert (sqllm_experts)."""
    _fields_ = [("packed", _vp), ("lut", _vp), ("row_ptr", _vp), ("col_idx", _vp), ("val", _vp), ("nnz", _i64)]


_ep = ctypes.POINTER(Experts)
_lib.sqllm_moe_workspace_bytes.restype = _sz
_lib.sqllm_moe_workspace_bytes.argtypes = [_i32, _i32, _i32, _i64, _i64]
_lib.sqllm_moe_route.restype = _i32
_lib.sqllm_moe_route.argtypes = [_vp, _vp, _vp, _i32, _i32, _i64, _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp]
_lib.sqllm_moe_experts.restype = _i32
_lib.sqllm_moe_experts.argtypes = [_vp, _vp, _vp, _ep, _ep, _ep, _i32, _i32, _i32, _i32, _i64, _i64, _vp, _vp, _sz, _vp]
_lib.sqllm_moe_layer.restype = _i32
_lib.sqllm_moe_layer.argtypes = [_vp, _vp, _vp, _i32, _f32, _ep, _ep, _ep, _i32, _i32, _i32, _i32, _i64, _i64, _vp, _vp,
                                 _vp, _vp, _sz, _vp]

EXPORTS = ("sqllm_moe_workspace_bytes", "sqllm_moe_route", "sqllm_moe_experts", "sqllm_moe_layer")
_SIGMOID, _KEEP_SUM = 1, 2
_MAX_TOPK, _ERR_SHAPE = 8, 3
_route, _experts, _layer = _lib.sqllm_moe_route, _lib.sqllm_moe_experts, _lib.sqllm_moe_layer


@functools.lru_cache(maxsize=4096)
def moe_workspace_bytes(batch: int, experts: int, topk: int, hidden: int, inter: int) -> int:
    if not (_calls.held(_i32, batch, experts, topk) and _calls.held(_i64, hidden, inter)):
        return 0
    return int(_lib.sqllm_moe_workspace_bytes(batch, experts, topk, hidden, inter))


_packed_bytes = functools.lru_cache(maxsize=4096)(packed_bytes)


def _projection(p, name, bits, rows, cols, experts, index) -> Experts:
    packed, lut = p["packed"], p["lut"]
    if lut.shape != (experts, rows, 1 << bits):
        raise ValueError(f"{name}.lut: shape {(experts, rows, 1 << bits)} expected, got {tuple(lut.shape)}")
    need = experts * _packed_bytes(rows, cols, bits)
    if packed.numel() < need or need == 0:
        raise ValueError(f"{name}.packed: {need} bytes expected, got {packed.numel()}")
    pp, lp = _calls.address(packed, f"{name}.packed", torch.uint8, index), _calls.address(lut, f"{name}.lut", torch.float16, index)
    col = p.get("col")
    if col is None or col.numel() == 0:
        return Experts(pp, lp, None, None, None, 0)
    row_ptr, val, nnz = p["row_ptr"], p["val"], col.numel()
    if row_ptr.numel() != experts * rows + 1 or val.numel() != nnz:
        raise ValueError(f"{name}: row_ptr of {experts * rows + 1} entries and as many values as columns expected")
    return Experts(pp, lp, _calls.address(row_ptr, f"{name}.row_ptr", torch.int32, index),
                   _calls.address(col, f"{name}.col", torch.uint16 if col.dtype is torch.uint16 else torch.int16, index),
                   _calls.address(val, f"{name}.val", torch.float16, index), nnz)


def _projections(gate, up, down, bits, experts, hidden, inter, index):
    return (_projection(gate, "gate", bits, inter, hidden, experts, index),
            _projection(up, "up", bits, inter, hidden, experts, index),
            _projection(down, "down", bits, hidden, inter, experts, index))


def _rows_of(x):
    if x.dim() != 2:
        raise ValueError(f"x: shape (batch, hidden) expected, got {tuple(x.shape)}")
    return x.shape


def _router(x, router, bias, topk, index, call):
    batch, hidden = _rows_of(x)
    if not 0 < topk <= _MAX_TOPK:  # before outputs of that width are made
        _check(_ERR_SHAPE, call)
    rp = _calls.address(router, "router", torch.float16, index)
    if router.dim() != 2 or router.shape[1] != hidden:
        raise ValueError(f"router: shape (experts, {hidden}) expected, got {tuple(router.shape)}")
    experts = router.shape[0]
    if bias is None:
        return batch, hidden, experts, rp, None
    if bias.shape != (experts,):
        raise ValueError(f"bias: shape {(experts,)} expected, got {tuple(bias.shape)}")
    return batch, hidden, experts, rp, _calls.address(bias, "bias", torch.float32, index)


@_calls.on_stream
def moe_route(index, handle, x: torch.Tensor, router: torch.Tensor, topk: int, bias: torch.Tensor | None = None, sigmoid: bool = False,
              renormalize: bool = True, scale: float = 1.0, ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """(ids int32, weights fp32), both [batch, topk]: each token's experts by softmax (or sigmoid) scores of
    x router^T.  bias (fp32 [experts]) moves the choice only; renormalize divides a token's weights by their sum.
    stream: as for every call (keyword)."""
    batch, hidden, experts, rp, bp = _router(x, router, bias, topk, index, "sqllm_moe_route")
    xp = _calls.address(x, "x", torch.float16, index)
    flags = (_SIGMOID if sigmoid else 0) | (0 if renormalize else _KEEP_SUM)
    ids, ip = _calls.output(ids, "ids", (batch, topk), torch.int32, index)
    weights, wp = _calls.output(weights, "weights", (batch, topk), torch.float32, index)
    _check(_calls.with_scratch(
        ws, moe_workspace_bytes(batch, experts, topk, hidden, 256), index, handle, _route, xp, rp, bp, batch, experts,
        hidden, topk, flags, scale, ip, wp), "sqllm_moe_route")
    return ids, weights


@_calls.on_stream
def moe_experts(index, handle, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate: dict, up: dict, down: dict, bits: int,
                y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """y [batch, hidden] = sum over a token's ids of weight * down(silu(gate x) * up x).  An id outside
    [0, experts) (-1 for a padded row) takes no part; a token without any gets zeros."""
    batch, hidden = _rows_of(x)
    ip, wp = _calls.address(ids, "ids", torch.int32, index), _calls.address(weights, "weights", torch.float32, index)
    if ids.dim() != 2 or ids.shape[0] != batch or weights.shape != ids.shape:
        raise ValueError(f"ids, weights: shape ({batch}, topk) expected, got {tuple(ids.shape)}, {tuple(weights.shape)}")
    topk, (experts, inter) = ids.shape[1], gate["lut"].shape[:2]
    g, u, d = _projections(gate, up, down, bits, experts, hidden, inter, index)
    xp = _calls.address(x, "x", torch.float16, index)
    y, yp = _calls.output(y, "y", (batch, hidden), torch.float16, index)
    _check(_calls.with_scratch(
        ws, moe_workspace_bytes(batch, experts, topk, hidden, inter), index, handle, _experts, xp, ip, wp, g, u, d, bits,
        batch, experts, topk, hidden, inter, yp), "sqllm_moe_experts")
    return y


@_calls.on_stream
def moe_layer(index, handle, x: torch.Tensor, router: torch.Tensor, topk: int, gate: dict, up: dict, down: dict, bits: int,
              bias: torch.Tensor | None = None, sigmoid: bool = False, renormalize: bool = True, scale: float = 1.0,
              y: torch.Tensor | None = None, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
              ws: torch.Tensor | None = None):
    """(y, ids, weights): moe_route and moe_experts in one call."""
    batch, hidden, experts, rp, bp = _router(x, router, bias, topk, index, "sqllm_moe_layer")
    inter = gate["lut"].shape[1]
    g, u, d = _projections(gate, up, down, bits, experts, hidden, inter, index)
    xp = _calls.address(x, "x", torch.float16, index)
    flags = (_SIGMOID if sigmoid else 0) | (0 if renormalize else _KEEP_SUM)
    y, yp = _calls.output(y, "y", (batch, hidden), torch.float16, index)
    ids, ip = _calls.output(ids, "ids", (batch, topk), torch.int32, index)
    weights, wp = _calls.output(weights, "weights", (batch, topk), torch.float32, index)
    _check(_calls.with_scratch(
        ws, moe_workspace_bytes(batch, experts, topk, hidden, inter), index, handle, _layer, xp, rp, bp, flags, scale, g, u,
        d, bits, batch, experts, topk, hidden, inter, ip, wp, yp), "sqllm_moe_layer")
    return y, ids, weights
