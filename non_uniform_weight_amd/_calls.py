"""What the calls with plain scratch share: the stream and device a call runs on, and its scratch.

Unlike the products' workspace, this scratch need not be zero and is left with any contents, so it is kept apart
from theirs.  It is cached per (device, stream); the launches of one call follow each other on the stream, so one
buffer serves every call there.  A call under graph capture takes a buffer of its own from the graph's memory:
replays of two graphs, or of a graph beside eager calls, never meet in one buffer."""
from __future__ import annotations

import contextlib
import threading

import torch

_SCRATCH: dict = {}
# Several host threads may call on one stream: the launches of a call that uses the stream's buffer may not be
# interleaved with another's.
LOCK = threading.Lock()


def one_device(tensors) -> torch.device:
    """The device that every tensor given is on (None entries are skipped)."""
    dev = None
    for name, t in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: torch.Tensor expected")
        if not t.is_cuda:
            raise ValueError(f"{name}: device tensor expected (the operators run only on the GPU)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name}: on {t.device}, the other tensors on {dev}")
    return dev


def on(device: torch.device, stream):
    """Context in which `device` is current and work goes to `stream` (None: the device's current stream)."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream: on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return contextlib.nullcontext()


def scratch(nbytes: int, device: torch.device, handle: int) -> torch.Tensor:
    """Scratch for a call on the current stream, whose handle is given (LOCK held)."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, handle)
    buf = _SCRATCH.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = _SCRATCH[key] = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
    return buf
