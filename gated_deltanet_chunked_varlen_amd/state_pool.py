"""Python binding of the state-pool row operators (include/gdn_prefill.h,
gdn_pool_*): rows copied or forked, zeroed, compacted.

A pool is any tensor whose first dimension counts rows and whose other one to
three dimensions are a state: [rows, H, V, K] of ``chunk_gated_delta_rule``,
[rows, H, D] of ``gated_linear_recurrence``, or [rows, n].  Views are taken as
they are (a layer's slice of a [rows, layers, ...] pool).  Row lists are int32
or int64 device tensors; an entry of -1 is padding.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as nat
from .api import _STATE_DTYPES, _index, _ptr, _raise, state_tensor


def _pool_fields(name, pool, written):
    """(tensor, dtype, rows, strides[4], extent[3]) of a pool."""
    if not isinstance(pool, torch.Tensor) or not pool.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not 2 <= pool.dim() <= 4:
        raise ValueError("%s must be [rows, ...] with one to three state dimensions" % name)
    if pool.dtype not in _STATE_DTYPES:
        raise ValueError("unsupported %s dtype" % name)
    if any(n == 0 for n in pool.shape[1:]):
        raise ValueError("%s has empty rows" % name)
    pool = state_tensor(name, pool, written)
    pad = 4 - pool.dim()
    extent = (1,) * pad + tuple(pool.shape[1:])
    # a dimension of extent 1 is never stepped over; 1 keeps all-zero strides
    # (contiguous in the C ABI) out
    strides = [st if n > 1 else 1 for n, st in zip(pool.shape, pool.stride())]
    strides = [strides[0]] + [1] * pad + strides[1:]
    return pool, _STATE_DTYPES[pool.dtype], pool.shape[0], nat._i64x4(*strides), extent


def _list(name, rows, device):
    if not isinstance(rows, torch.Tensor) or rows.device != device:
        raise ValueError("%s must be a tensor on %s" % (name, device))
    return _index(name, rows)


def _params(pool, dst_rows, status):
    pool, dtype, rows, strides, extent = _pool_fields("pool", pool, True)
    p = nat.PoolParams()
    p.extent = nat._i64x3(*extent)
    p.dst, p.dst_dtype, p.dst_pool_rows, p.dst_strides = _ptr(pool), dtype, rows, strides
    if status is not None:
        if status.device != pool.device or status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError("status must be an int32 tensor on %s" % pool.device)
        p.status = _ptr(status)
    p.dst_rows, p.count = _ptr(dst_rows), dst_rows.numel()
    return p


def _call(fn, p, device, *more):
    with torch.cuda.device(device):
        stream = torch.cuda.current_stream(device).cuda_stream
        rc = fn(ctypes.byref(p), *more, ctypes.c_void_p(stream))
    if rc != 0:
        _raise(rc)


def state_pool_copy(pool, src_rows, dst_rows, src_pool=None, status=None):
    """pool[dst_rows[i]] = src_pool[src_rows[i]] for every i, on the current
    stream: a row forked into several, moved, or brought in from another pool
    or a checkpoint buffer (src_pool, any state dtype; None: pool itself).

    Equal dtypes copy bit for bit, others round to nearest (8-bit types
    saturate).  A destination named twice takes its last entry; inside one
    pool an entry whose source row is another entry's destination is skipped;
    entries outside the pools are skipped.  ``status`` (optional int32 device
    tensor) receives the matching GDN_STATUS_POOL_* bits.  src_pool may be the
    same view as pool, or share no elements with it.  Returns pool."""
    device = pool.device if isinstance(pool, torch.Tensor) else None
    kind = _list("src_rows", src_rows, device)
    if _list("dst_rows", dst_rows, device) != kind:
        raise ValueError("src_rows and dst_rows must share a dtype")
    if src_rows.numel() != dst_rows.numel():
        raise ValueError("src_rows and dst_rows must have the same length")
    p = _params(pool, dst_rows, status)
    p.rows_type, p.src_rows = kind, _ptr(src_rows)
    src = pool if src_pool is None else src_pool
    src, p.src_dtype, p.src_pool_rows, p.src_strides, extent = _pool_fields("src_pool", src, False)
    if src.device != device:
        raise ValueError("src_pool must be on %s" % device)
    if tuple(extent) != tuple(p.extent):
        raise ValueError("rows of pool and src_pool differ in shape")
    p.src = _ptr(src)
    if pool.shape[0] == 0 or src.shape[0] == 0:
        if src_rows.numel() > 0:
            raise ValueError("a pool without rows cannot be copied from or into")
        return pool
    _call(nat.lib().gdn_pool_copy, p, device)
    return pool


def state_pool_reset(pool, rows, status=None):
    """pool[rows[i]] = 0 for every i, on the current stream: rows freed, or
    taken for sequences that start from zero.  Entries outside the pool are
    skipped and set GDN_STATUS_POOL_ROW in ``status``.  Returns pool."""
    device = pool.device if isinstance(pool, torch.Tensor) else None
    kind = _list("rows", rows, device)
    p = _params(pool, rows, status)
    p.rows_type = kind
    _call(nat.lib().gdn_pool_reset, p, device)
    return pool


def state_pool_compact(pools, state_indices, output_indices=None, row_map=None, status=None):
    """Moves the live rows of a pool, the ones state_indices names, to its
    front, on the current stream and without a look at the host.

    With m distinct live rows, the k-th live row at or behind row m
    (ascending) is copied to the k-th row before m that is not live; no other
    row changes, so rows at or behind m can be dropped or reused.  ``pools`` is
    one pool or a list of pools with the same number of rows and the same use
    of them (the layers of a model), all moved alike.  Returns (state_indices
    with the moved rows renamed, num_live int32 [1]); output_indices, if given,
    receives the renamed list and must not overlap state_indices.  row_map
    (int32 [rows]) receives each row's new place, -1 for rows not live.
    Invalid entries stay as they are and set GDN_STATUS_POOL_ROW."""
    pools = list(pools) if isinstance(pools, (list, tuple)) else [pools]
    if not pools:
        raise ValueError("state_pool_compact needs a pool")
    device = pools[0].device if isinstance(pools[0], torch.Tensor) else None
    kind = _list("state_indices", state_indices, device)
    if output_indices is None:
        output_indices = torch.empty_like(state_indices)
    elif (output_indices.device != device or output_indices.dtype != state_indices.dtype
          or output_indices.shape != state_indices.shape or not output_indices.is_contiguous()):
        raise ValueError("output_indices must match state_indices")
    if row_map is not None and (row_map.device != device or row_map.dtype != torch.int32
                                or tuple(row_map.shape) != (pools[0].shape[0],)
                                or not row_map.is_contiguous()):
        raise ValueError("row_map must be contiguous int32 [%d] on %s"
                         % (pools[0].shape[0], device))
    calls = []
    for pool in pools:
        p = _params(pool, state_indices, status)
        if pool.device != device or pool.shape[0] != pools[0].shape[0]:
            raise ValueError("pools must share a device and a number of rows")
        p.rows_type = kind
        calls.append(p)
    num_live = torch.empty(1, dtype=torch.int32, device=device)
    for p in calls:
        _call(nat.lib().gdn_pool_compact, p, device, _ptr(output_indices), _ptr(num_live),
              _ptr(row_map))
    return output_indices, num_live
