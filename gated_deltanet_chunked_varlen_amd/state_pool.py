"""Python binding of the state-pool row operators (include/gdn_prefill.h,
gdn_pool_*): rows copied or forked, zeroed, compacted.

A pool is any tensor whose first dimension counts rows and whose other one to
three dimensions are a state: [rows, H, V, K] of ``chunk_gated_delta_rule``,
[rows, H, D] of ``gated_linear_recurrence``, or [rows, n].  Views are taken as
they are (a layer's slice of a [rows, layers, ...] pool).  Row lists are int32
or int64 device tensors; an entry of -1 is padding.  As with torch's in-place
operators a pool must not require a gradient (but under torch.no_grad()), and
its autograd version advances.  No call is differentiable: a src_pool that
requires a gradient is refused too.
"""
from __future__ import annotations

from ._launch import calls


def state_pool_copy(pool, src_rows, dst_rows, src_pool=None, status=None):
    """pool[dst_rows[i]] = src_pool[src_rows[i]] for every i, on the current
    stream: a row forked into several, moved, or brought in from another pool
    or a checkpoint buffer (src_pool, any state dtype; None: pool itself).

    Equal dtypes copy bit for bit, others round to nearest (8-bit types
    saturate).  A destination named twice takes its last entry; inside one
    pool an entry whose source row is another entry's destination is skipped,
    unless that one copies the row onto itself (src [0, 0], dst [0, 1] keeps
    row 0 and forks it; a swap is skipped both ways);
    entries outside the pools are skipped.  A list holds at most 262144
    entries; it is meant for a few thousand (each is compared with all
    others).  ``status`` (optional int32 device
    tensor) receives the matching GDN_STATUS_POOL_* bits.  src_pool may be the
    same view as pool, or share no elements with it (views whose address
    ranges cross need equal strides).  Returns pool."""
    return calls().pool_copy(pool, src_rows, dst_rows, src_pool, status)


def state_pool_reset(pool, rows, status=None):
    """pool[rows[i]] = 0 for every i, on the current stream: rows freed, or
    taken for sequences that start from zero.  Entries outside the pool are
    skipped and set GDN_STATUS_POOL_ROW in ``status``.  Returns pool."""
    return calls().pool_reset(pool, rows, status)


def state_pool_compact(pools, state_indices, output_indices=None, row_map=None, status=None):
    """Moves the live rows of a pool, the ones state_indices names, to its
    front, on the current stream and without a look at the host.

    With m distinct live rows, the k-th live row at or behind row m
    (ascending) is copied to the k-th row before m that is not live; no other
    row changes, so rows at or behind m can be dropped or reused.  ``pools`` is
    one pool or a list of pools with the same number of rows and the same use
    of them (the layers of a model), all moved alike, or none if one of them is
    refused.  Returns (state_indices
    with the moved rows renamed, num_live int32 [1]); output_indices, if given,
    receives the renamed list and must not overlap state_indices.  row_map
    (int32 [rows]) receives each row's new place, -1 for rows not live.
    Invalid entries stay as they are and set GDN_STATUS_POOL_ROW."""
    pools = list(pools) if isinstance(pools, (list, tuple)) else [pools]
    return calls().pool_compact(pools, state_indices, output_indices, row_map, status)
