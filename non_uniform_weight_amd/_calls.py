"""What the calls with plain scratch share: checked addresses, the stream and device a call runs on, and its scratch.

Unlike the products' workspace, this scratch need not be zero and is left with any contents, so it is kept apart
from theirs.  It is cached per (device, stream); the launches of one call follow each other on the stream, so one
buffer serves every call there.  A call under graph capture takes a buffer of its own from the graph's memory:
replays of two graphs, or of a graph beside eager calls, never meet in one buffer.

Small calls take a few microseconds on the GPU, so the checks here are the cheapest that tell the same."""
from __future__ import annotations

import functools
import inspect
import threading

import torch


def held(ctype, *values: int) -> bool:
    """Whether the C type holds the values: ctypes cuts larger ones to their low bits without a word."""
    return all(ctype(v).value == v for v in values)


_SCRATCH: dict = {}
# Several host threads may call on one stream: the launches of a call that uses the stream's buffer may not be
# interleaved with another's.
_LOCK = threading.Lock()


def device_of(x, name: str) -> int:
    """Index of the device that x is on; the call's other tensors have to be there too."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected")
    index = x.get_device()
    if index < 0:
        raise ValueError(f"{name}: device tensor expected (the operators run only on the GPU)")
    return index


def address(t, name: str, dtype, index: int) -> int:
    """Address of a contiguous tensor of this type on device `index`."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _checked_address(t, name, dtype, index)


def _checked_address(t, name: str, dtype, index: int) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected")
    if t.get_device() < 0:
        raise ValueError(f"{name}: device tensor expected (the operators run only on the GPU)")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the call's other tensors on cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {dtype} expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    return t.data_ptr()


def half_rows(x, name: str, index: int):
    """(rows, columns, values from a row to the next, address) of fp16 x [rows, cols], its columns adjacent."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected")
    shape = x.shape
    if len(shape) != 2 or 0 in shape:
        raise ValueError(f"{name}: shape (rows, cols) expected, got {tuple(shape)}")
    if x.dtype is not torch.float16 or x.get_device() != index:
        _checked_address(x, name, torch.float16, index)
    rows, cols = shape
    if x.is_contiguous():
        return rows, cols, cols, x.data_ptr()
    if cols > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: adjacent columns expected")
    return rows, cols, x.stride(0) if rows > 1 else cols, x.data_ptr()


def output(t, name: str, shape: tuple, dtype, index: int):
    """(t, its address); a new tensor where t is None.  Called with the call's stream current."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=index)
        return t, t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name}: shape {shape} expected, got {tuple(t.shape)}")
    return t, address(t, name, dtype, index)


_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def on_stream(fn):
    """Runs fn(index, handle, ...) with the device of its first tensor current and its keyword `stream`, if given, as
    the current stream; handle is that stream's."""

    # what a caller sees: fn's arguments but the first two, and stream
    mine = inspect.signature(fn)
    rest = [p for p in mine.parameters.values()][2:]
    name = rest[0].name

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        index = device_of(args[0] if args else kw.get(name), name)
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"stream: on {stream.device}, the tensors on cuda:{index}")
            with torch.cuda.stream(stream):
                return fn(index, stream.cuda_stream, *args, **kw)
        if _device() != index:
            with torch.cuda.device(index):
                return fn(index, _raw_stream(index), *args, **kw)
        return fn(index, _raw_stream(index), *args, **kw)

    call.__signature__ = mine.replace(parameters=[*rest, inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def with_scratch(ws, nbytes: int, index: int, handle: int, fn, *args) -> int:
    """fn(*args, address, bytes, handle) with ws (uint8 tensor) or, if None, scratch of the current stream."""
    if ws is not None:
        return fn(*args, address(ws, "workspace", torch.uint8, index), ws.numel(), handle)
    if torch._C._cuda_isCurrentStreamCapturing():
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=index)
        return fn(*args, ws.data_ptr(), ws.numel(), handle)
    with _LOCK:
        buf = _SCRATCH.get((index, handle))
        if buf is None or buf[1] < nbytes:
            ws = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=index)
            buf = _SCRATCH[index, handle] = (ws.data_ptr(), ws.numel(), ws)
        return fn(*args, buf[0], buf[1], handle)
