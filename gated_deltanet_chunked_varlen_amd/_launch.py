"""Cheap repeated calls for the bindings of small operators.

A decode step or a row copy runs for a few microseconds on the GPU, less than
checking its arguments from Python takes.  The checks depend on the arguments'
shapes, strides, types and devices alone, so a call keeps its filled parameter
block (without addresses) under exactly those and, when they come again, only
puts the addresses in.  What depends on an address (alignment, overlap) the C
ABI checks on every call.
"""
from __future__ import annotations

import torch

from . import api

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else None


def meta(t):
    """What the checks read of an optional tensor."""
    if t is None:
        return None
    try:
        return (t.shape, t.stride(), t.dtype, t.device)
    except AttributeError:
        raise ValueError("a tensor is expected, not %s" % type(t).__name__) from None


class Blocks:
    """Checked parameter blocks by the call's metadata, at most ``limit``
    (beyond, all are dropped: a program with that many shapes gains nothing)."""

    def __init__(self, struct, limit=512):
        self.struct, self.limit = struct, limit
        self._kept = {}

    def get(self, key):
        """(a fresh copy of the block, what was kept beside it), or None."""
        hit = self._kept.get(key)
        return None if hit is None else (self.struct.from_buffer_copy(hit[0]), hit[1])

    def keep(self, key, block, beside=None):
        """Keeps the block as it is now; call it before addresses go in."""
        if len(self._kept) >= self.limit:
            self._kept.clear()
        self._kept[key] = (bytes(block), beside)


def current_stream(index):
    """Handle of the current stream of a device."""
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def call(fn, device, *args):
    """fn(*args, stream) with ``device`` current, on its current stream;
    raises on an error code."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, current_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, current_stream(index))
    if rc != 0:
        api._raise(rc)


def workspace(device, need):
    """Memory for a call on the device's current stream: kept per stream, or
    under capture from the graph's own pool (a graph keeps the address)."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=device)
    stream = current_stream(device.index)
    ws = api._ws_cache.get((device.type, device.index, stream))
    return ws if ws is not None and ws.numel() >= need else \
        api.cached_workspace(device, stream, need)

