"""Python binding of the state-pool row operators (include/gdn_prefill.h,
gdn_pool_*): rows copied or forked, zeroed, compacted.

A pool is any tensor whose first dimension counts rows and whose other one to
three dimensions are a state: [rows, H, V, K] of ``chunk_gated_delta_rule``,
[rows, H, D] of ``gated_linear_recurrence``, or [rows, n].  Views are taken as
they are (a layer's slice of a [rows, layers, ...] pool).  Row lists are int32
or int64 device tensors; an entry of -1 is padding.
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import _launch
from . import _native as nat
from ._launch import Blocks, meta
from .api import _STATE_DTYPES, _index, state_tensor


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


def _tensors(*args):
    return all(isinstance(t, torch.Tensor) for t in args)


def _list(name, rows, device):
    if not isinstance(rows, torch.Tensor) or rows.device != device:
        raise ValueError("%s must be a tensor on %s" % (name, device))
    return _index(name, rows)


def _check_status(status, device):
    if status is not None and (status.device != device or status.dtype != torch.int32
                               or status.numel() < 1):
        raise ValueError("status must be an int32 tensor on %s" % device)


def _block(pool, kind, count):
    """Parameter block of a call on ``pool``, without addresses."""
    _, dtype, rows, strides, extent = _pool_fields("pool", pool, True)
    p = nat.PoolParams()
    p.extent = nat._i64x3(*extent)
    p.dst_dtype, p.dst_pool_rows, p.dst_strides = dtype, rows, strides
    p.rows_type, p.count = kind, count
    return p


_int32_like = {}


def _one_int32(device):
    """A new int32 [1]; made after a pattern, which costs half of torch.empty."""
    like = _int32_like.get(device)
    if like is None:
        like = _int32_like[device] = torch.empty(1, dtype=torch.int32, device=device)
    return torch.empty_like(like)


_copy_blocks = Blocks(nat.PoolParams)
_reset_blocks = Blocks(nat.PoolParams)
_compact_blocks = Blocks(nat.PoolParams)


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
    src = pool if src_pool is None else src_pool
    key = (meta(pool), meta(src_rows), meta(dst_rows), meta(src_pool), meta(status)) \
        if _tensors(pool, src_rows, dst_rows, src) else None
    hit = _copy_blocks.get(key)
    if hit is None:
        device = pool.device if isinstance(pool, torch.Tensor) else None
        kind = _list("src_rows", src_rows, device)
        if _list("dst_rows", dst_rows, device) != kind:
            raise ValueError("src_rows and dst_rows must share a dtype")
        if src_rows.numel() != dst_rows.numel():
            raise ValueError("src_rows and dst_rows must have the same length")
        _check_status(status, device)
        p = _block(pool, kind, dst_rows.numel())
        read, p.src_dtype, p.src_pool_rows, p.src_strides, extent = _pool_fields(
            "src_pool", src, False)
        if src.device != device:
            raise ValueError("src_pool must be on %s" % device)
        if tuple(extent) != tuple(p.extent):
            raise ValueError("rows of pool and src_pool differ in shape")
        if src_rows.numel() > 0 and (pool.shape[0] == 0 or src.shape[0] == 0):
            raise ValueError("a pool without rows cannot be copied from or into")
        if read is src:
            _copy_blocks.keep(key, p)
        src = read
    else:
        p = hit[0]
    if pool.shape[0] == 0 or src.shape[0] == 0:
        return pool
    p.src, p.dst = src.data_ptr(), pool.data_ptr()
    p.src_rows, p.dst_rows = src_rows.data_ptr(), dst_rows.data_ptr()
    if status is not None:
        p.status = status.data_ptr()
    _launch.call(nat.lib().gdn_pool_copy, pool.device, byref(p))
    return pool


def state_pool_reset(pool, rows, status=None):
    """pool[rows[i]] = 0 for every i, on the current stream: rows freed, or
    taken for sequences that start from zero.  Entries outside the pool are
    skipped and set GDN_STATUS_POOL_ROW in ``status``.  Returns pool."""
    key = (meta(pool), meta(rows), meta(status)) if _tensors(pool, rows) else None
    hit = _reset_blocks.get(key)
    if hit is None:
        device = pool.device if isinstance(pool, torch.Tensor) else None
        kind = _list("rows", rows, device)
        _check_status(status, device)
        p = _block(pool, kind, rows.numel())
        _reset_blocks.keep(key, p)
    else:
        p = hit[0]
    p.dst, p.dst_rows = pool.data_ptr(), rows.data_ptr()
    if status is not None:
        p.status = status.data_ptr()
    _launch.call(nat.lib().gdn_pool_reset, pool.device, byref(p))
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
    blocks = []
    for pool in pools:
        key = (meta(pool), meta(state_indices), meta(output_indices), meta(row_map),
               meta(status), meta(pools[0])) if _tensors(pool, state_indices) else None
        hit = _compact_blocks.get(key)
        if hit is None:
            kind = _list("state_indices", state_indices, device)
            if output_indices is not None and (
                    output_indices.device != device
                    or output_indices.dtype != state_indices.dtype
                    or output_indices.shape != state_indices.shape
                    or not output_indices.is_contiguous()):
                raise ValueError("output_indices must match state_indices")
            if row_map is not None and (row_map.device != device or row_map.dtype != torch.int32
                                        or tuple(row_map.shape) != (pools[0].shape[0],)
                                        or not row_map.is_contiguous()):
                raise ValueError("row_map must be contiguous int32 [%d] on %s"
                                 % (pools[0].shape[0], device))
            _check_status(status, device)
            p = _block(pool, kind, state_indices.numel())
            if pool.device != device or pool.shape[0] != pools[0].shape[0]:
                raise ValueError("pools must share a device and a number of rows")
            _compact_blocks.keep(key, p)
        else:
            p = hit[0]
        blocks.append(p)
    if output_indices is None:
        output_indices = torch.empty_like(state_indices)
    num_live = _one_int32(device)
    for pool, p in zip(pools, blocks):
        p.dst, p.dst_rows = pool.data_ptr(), state_indices.data_ptr()
        if status is not None:
            p.status = status.data_ptr()
        _launch.call(nat.lib().gdn_pool_compact, device, byref(p), output_indices.data_ptr(),
                     num_live.data_ptr(), None if row_map is None else row_map.data_ptr())
    return output_indices, num_live
