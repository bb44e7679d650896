"""A mixture-of-experts layer for up to 16 tokens whose experts are dense-and-sparse LUT matrices
(include/sqllm_moe.h): the router's choice, the experts' products, and both as one call.

A projection of the experts is a dict like a group product's item, over all experts: packed (the experts' packed
matrices one after another), lut (fp16 [experts, rows, 2^bits]) and, with outliers, one CSR over the experts' rows:
row_ptr (int32 [experts * rows + 1]), col (uint16 or int16 bits), val (fp16)."""
from __future__ import annotations

import ctypes

import torch

from . import _calls, _check, _csr_ptrs, _dev, _lib, packed_bytes

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


def moe_workspace_bytes(batch: int, experts: int, topk: int, hidden: int, inter: int) -> int:
    return int(_lib.sqllm_moe_workspace_bytes(batch, experts, topk, hidden, inter))


def _out(t, name, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {shape} expected, got {tuple(t.shape)}")
    return t


def _rows_of(x):
    if x.dim() != 2:
        raise ValueError(f"x: shape (batch, hidden) expected, got {tuple(x.shape)}")
    return x.shape


def _projection(p, name, bits, rows, cols, experts) -> Experts:
    lut = p["lut"]
    if tuple(lut.shape) != (experts, rows, 1 << bits):
        raise ValueError(f"{name}.lut: shape {(experts, rows, 1 << bits)} expected, got {tuple(lut.shape)}")
    need = experts * packed_bytes(rows, cols, bits)
    if p["packed"].numel() < need or need == 0:
        raise ValueError(f"{name}.packed: {need} bytes expected, got {p['packed'].numel()}")
    rp, ci, cv, nnz = _csr_ptrs(p.get("row_ptr"), p.get("col"), p.get("val"))
    if nnz and (p["row_ptr"].numel() != experts * rows + 1 or p["val"].numel() != nnz):
        raise ValueError(f"{name}: row_ptr of {experts * rows + 1} entries and as many values as columns expected")
    return Experts(_dev(p["packed"], f"{name}.packed", torch.uint8), _dev(lut, f"{name}.lut", torch.float16), rp, ci, cv,
                   nnz)


def _projections(gate, up, down, bits, experts, hidden, inter):
    return (_projection(gate, "gate", bits, inter, hidden, experts), _projection(up, "up", bits, inter, hidden, experts),
            _projection(down, "down", bits, hidden, inter, experts))


def _named(gate, up, down):
    return tuple((f"{n}.{k}", p.get(k)) for n, p in (("gate", gate), ("up", up), ("down", down))
                 for k in ("packed", "lut", "row_ptr", "col", "val"))


def _router(x, router, topk, bias):
    batch, hidden = _rows_of(x)
    if router.dim() != 2 or router.shape[1] != hidden:
        raise ValueError(f"router: shape (experts, {hidden}) expected, got {tuple(router.shape)}")
    experts = router.shape[0]
    if bias is not None and tuple(bias.shape) != (experts,):
        raise ValueError(f"bias: shape {(experts,)} expected, got {tuple(bias.shape)}")
    return batch, hidden, experts


def moe_route(x: torch.Tensor, router: torch.Tensor, topk: int, bias: torch.Tensor | None = None, sigmoid: bool = False,
              renormalize: bool = True, scale: float = 1.0, ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """(ids int32, weights fp32), both [batch, topk]: each token's experts by softmax (or sigmoid) scores of
    x router^T.  bias (fp32 [experts]) moves the choice only; renormalize divides a token's weights by their sum."""
    dev = _calls.one_device((("x", x), ("router", router), ("bias", bias), ("ids", ids), ("weights", weights),
                             ("workspace", ws)))
    batch, hidden, experts = _router(x, router, topk, bias)
    with _calls.on(dev, stream):
        ids = _out(ids, "ids", (batch, topk), torch.int32, dev)
        weights = _out(weights, "weights", (batch, topk), torch.float32, dev)
        handle = torch.cuda.current_stream().cuda_stream
        with _calls.LOCK:
            buf = _calls.scratch(moe_workspace_bytes(batch, experts, topk, hidden, 256), dev, handle) if ws is None else ws
            _check(_lib.sqllm_moe_route(
                _dev(x, "x", torch.float16), _dev(router, "router", torch.float16),
                None if bias is None else _dev(bias, "bias", torch.float32), batch, experts, hidden, topk,
                (_SIGMOID if sigmoid else 0) | (0 if renormalize else _KEEP_SUM), scale, _dev(ids, "ids", torch.int32),
                _dev(weights, "weights", torch.float32), _dev(buf, "workspace", torch.uint8), buf.numel(), handle),
                "sqllm_moe_route")
    return ids, weights


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate: dict, up: dict, down: dict, bits: int,
                y: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [batch, hidden] = sum over a token's ids of weight * down(silu(gate x) * up x).  An id outside
    [0, experts) (-1 for a padded row) takes no part; a token without any gets zeros."""
    dev = _calls.one_device((("x", x), ("ids", ids), ("weights", weights), ("y", y), ("workspace", ws),
                             *_named(gate, up, down)))
    batch, hidden = _rows_of(x)
    experts, inter = gate["lut"].shape[:2]
    if ids.dim() != 2 or ids.shape[0] != batch or weights.shape != ids.shape:
        raise ValueError(f"ids, weights: shape ({batch}, topk) expected, got {tuple(ids.shape)}, {tuple(weights.shape)}")
    topk = ids.shape[1]
    g, u, d = _projections(gate, up, down, bits, experts, hidden, inter)
    with _calls.on(dev, stream):
        y = _out(y, "y", (batch, hidden), torch.float16, dev)
        handle = torch.cuda.current_stream().cuda_stream
        with _calls.LOCK:
            buf = _calls.scratch(moe_workspace_bytes(batch, experts, topk, hidden, inter), dev, handle) if ws is None else ws
            _check(_lib.sqllm_moe_experts(
                _dev(x, "x", torch.float16), _dev(ids, "ids", torch.int32), _dev(weights, "weights", torch.float32), g, u, d,
                bits, batch, experts, topk, hidden, inter, _dev(y, "y", torch.float16), _dev(buf, "workspace", torch.uint8),
                buf.numel(), handle), "sqllm_moe_experts")
    return y


def moe_layer(x: torch.Tensor, router: torch.Tensor, topk: int, gate: dict, up: dict, down: dict, bits: int,
              bias: torch.Tensor | None = None, sigmoid: bool = False, renormalize: bool = True, scale: float = 1.0,
              y: torch.Tensor | None = None, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
              ws: torch.Tensor | None = None, stream=None):
    """(y, ids, weights): moe_route and moe_experts in one call."""
    dev = _calls.one_device((("x", x), ("router", router), ("bias", bias), ("y", y), ("ids", ids), ("weights", weights),
                             ("workspace", ws), *_named(gate, up, down)))
    batch, hidden, experts = _router(x, router, topk, bias)
    inter = gate["lut"].shape[1]
    g, u, d = _projections(gate, up, down, bits, experts, hidden, inter)
    with _calls.on(dev, stream):
        y = _out(y, "y", (batch, hidden), torch.float16, dev)
        ids = _out(ids, "ids", (batch, topk), torch.int32, dev)
        weights = _out(weights, "weights", (batch, topk), torch.float32, dev)
        handle = torch.cuda.current_stream().cuda_stream
        with _calls.LOCK:
            buf = _calls.scratch(moe_workspace_bytes(batch, experts, topk, hidden, inter), dev, handle) if ws is None else ws
            _check(_lib.sqllm_moe_layer(
                _dev(x, "x", torch.float16), _dev(router, "router", torch.float16),
                None if bias is None else _dev(bias, "bias", torch.float32),
                (_SIGMOID if sigmoid else 0) | (0 if renormalize else _KEEP_SUM), scale, g, u, d, bits, batch, experts,
                topk, hidden, inter, _dev(ids, "ids", torch.int32), _dev(weights, "weights", torch.float32),
                _dev(y, "y", torch.float16), _dev(buf, "workspace", torch.uint8), buf.numel(), handle), "sqllm_moe_layer")
    return y, ids, weights
