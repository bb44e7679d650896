"""What the calls with plain scratch share: checked addresses, the stream and device a call runs on, and its scratch.

Unlike the products' workspace, this scratch need not be zero and is left with any contents, so it is kept apart
from theirs.  It is cached per (device, stream); the launches of one call follow each other on the stream, so one
buffer serves every call there.  A call under graph capture takes a buffer of its own from the graph's memory:
replays of two graphs, or of a graph beside eager calls, never meet in one buffer.

Small calls take a few microseconds on the GPU, so the checks here are the cheapest that tell the same."""
from __future__ import annotations

import functools
import threading

import torch

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
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected")
    if t.get_device() != index:
        if t.get_device() < 0:
            raise ValueError(f"{name}: device tensor expected (the operators run only on the GPU)")
        raise ValueError(f"{name}: on {t.device}, the call's other tensors on cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {dtype} expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    return t.data_ptr()


def output(t, name: str, shape: tuple, dtype, index: int):
    """(t, its address); a new tensor where t is None.  Called with the call's stream current."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=index)
        return t, t.data_ptr()
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {shape} expected, got {tuple(t.shape)}")
    return t, address(t, name, dtype, index)


def on_stream(fn):
    """Runs fn(..., index, handle) with the device of its first tensor current and its keyword `stream`, if given, as
    the current stream; handle is that stream's."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        index = device_of(args[0] if args else next(iter(kw.values()), None), fn.__name__)
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"stream: on {stream.device}, the tensors on cuda:{index}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw, index=index, handle=stream.cuda_stream)
        if torch._C._cuda_getDevice() != index:
            with torch.cuda.device(index):
                return fn(*args, **kw, index=index, handle=torch._C._cuda_getCurrentRawStream(index))
        return fn(*args, **kw, index=index, handle=torch._C._cuda_getCurrentRawStream(index))

    return call


def with_scratch(ws, nbytes: int, index: int, handle: int, launch) -> int:
    """launch(address, bytes) with ws (uint8 tensor) or, if None, scratch of the current stream; its status."""
    if ws is not None:
        return launch(address(ws, "workspace", torch.uint8, index), ws.numel())
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=index)
        return launch(ws.data_ptr(), ws.numel())
    with _LOCK:
        buf = _SCRATCH.get((index, handle))
        if buf is None or buf.numel() < nbytes:
            buf = _SCRATCH[index, handle] = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=index)
        return launch(buf.data_ptr(), buf.numel())
