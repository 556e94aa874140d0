"""MI355X-native varlen chunked Gated Delta Rule prefill (libgdn_prefill).

``chunk_gated_delta_rule`` (with ``use_cp`` for context parallelism within
the GPU), ``chunk_gated_delta_rule_noalloc``, ``gated_delta_rule_decode`` and
``build_chunk_indices`` call the HIP kernels of the in-tree
``libgdn_prefill.so`` through its C ABI (include/gdn_prefill.h);
``PrefillGraphs`` replays one captured HIP graph per set of buffer addresses.

Beside the gated delta rule: ``gated_linear_recurrence`` (h = g h + x over the
same packed sequences, with its ``_backward`` and ``_decode``), and the rows of
a state pool, of either recurrence: ``state_pool_copy``, ``state_pool_reset``
and ``state_pool_compact``.
"""
from .api import (PrefillGraphs, build_chunk_indices, chunk_gated_delta_rule,  # noqa: F401
                  chunk_gated_delta_rule_noalloc, clear_workspace_cache,
                  gated_delta_rule_decode)
from .recurrence import (gated_linear_recurrence, gated_linear_recurrence_backward,  # noqa: F401
                         gated_linear_recurrence_decode)
from .state_pool import state_pool_compact, state_pool_copy, state_pool_reset  # noqa: F401

__all__ = ["chunk_gated_delta_rule", "chunk_gated_delta_rule_noalloc", "gated_delta_rule_decode",
           "build_chunk_indices", "PrefillGraphs", "clear_workspace_cache",
           "gated_linear_recurrence", "gated_linear_recurrence_backward",
           "gated_linear_recurrence_decode", "state_pool_copy", "state_pool_reset",
           "state_pool_compact"]
