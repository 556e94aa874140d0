"""The compiled marshalling of the recurrence, layer, beam and state-pool calls
(``_calls``, from csrc/torch_calls.cpp and torch_layer_calls.cpp), bound to the loaded library.

Both are built together; without either the calls raise ImportError.
"""
from __future__ import annotations

import ctypes
import threading
from collections import OrderedDict

import torch

from . import _native as nat
from . import api

_bound = None
_ws_cache: "OrderedDict[tuple, torch.Tensor]" = OrderedDict()
_ws_lock = threading.RLock()


def _stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _workspace(index, stream, need):
    """Workspace of a call on ``stream``, the current one of the current device
    ``index``: kept per stream, or under capture from the graph's own pool (a
    graph keeps the address).  The prefill's workspaces and their number are
    apart; of either kind those least recently used go first."""
    if torch.cuda.is_current_stream_capturing():
        return _memory(index, need)
    with _ws_lock:
        ws = _ws_cache.pop((index, stream), None)
        if ws is None or ws.numel() < need:
            ws = _memory(index, need)
        _ws_cache[index, stream] = ws
        while len(_ws_cache) > api._WS_CACHE_MAX:
            _ws_cache.popitem(last=False)
    return ws


def _memory(index, need):
    return torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index))


def calls():
    """The module of calls; raises if it or the library has not been built."""
    global _bound
    if _bound is None:
        lib = nat.lib()
        try:
            from . import _calls
        except ModuleNotFoundError:
            raise ImportError("_calls.so is not built; run "
                              "`python -m gated_deltanet_chunked_varlen_amd.build`") from None
        address = [ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "gdn_recurrence_workspace_size", "gdn_recurrence", "gdn_recurrence_backward",
            "gdn_recurrence_decode", "gdn_pool_copy", "gdn_pool_reset", "gdn_pool_compact",
            "gdn_validate_pool_host",
            "gdn_convolution_workspace_size", "gdn_convolution", "gdn_convolution_backward",
            "gdn_convolution_decode", "gdn_scan_chunk", "gdn_scan_workspace_size", "gdn_scan",
            "gdn_scan_backward", "gdn_scan_decode", "gdn_beam_workspace_size", "gdn_beam_select",
            "gdn_pool_reorder")]
        # torch's own accessor of the raw handle where it has one: a tenth of the time
        stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
        _calls.bind(*address, api._raise, stream, _workspace)
        _bound = _calls
    return _bound
