"""Python binding of beam search over recurrent states (include/gdn_prefill.h,
gdn_beam_select, gdn_pool_reorder): the best continuations of every group of
beams, and the rows of state pools brought in the order of their parents.

A recurrent state is overwritten with every token, so beams cannot share their
common past: a step selects (``beam_select``), and the pools' rows follow
(``state_pool_reorder``), one call for all layers.
"""
from __future__ import annotations

from ._launch import calls


def beam_select(logits, scores, num_candidates=None, workspace=None):
    """The best continuations of each group of beams, on the current stream.

    logits [batch, beams, vocabulary] float32, bfloat16 or float16 (a beam's
    values contiguous, beams evenly spaced), scores [batch, beams] float32, the
    beams' log probabilities so far.  Continuation v of beam k scores
    scores[k] + log_softmax(logits[k])[v]; the ``num_candidates`` best (None: as
    many as beams; at most 64, as the beams) of a group are returned best first,
    ties to the lowest beam, then the lowest token.  A beam that has ended is
    given the score -inf; its continuations, and tokens of logit -inf or NaN,
    come behind all others with the score -inf.  Scores are compared in 64 bits:
    those that are equal there are ties, whatever the logits.

    ``workspace`` (optional uint8 device tensor) is used, if it is large
    enough, instead of the one that is kept for the current stream.

    Returns (scores float32, parents int32, tokens int32), each [batch,
    num_candidates].  The call is not differentiable: tensors that require a
    gradient are refused (but under torch.no_grad())."""
    return calls().beam_select(logits, scores, num_candidates, workspace)


def state_pool_reorder(pools, state_indices, parents, output_indices=None, status=None):
    """Brings state pools in the order of the selected parents, on the current
    stream and without a look at the host.

    Beam k of group b holds row state_indices[b * beams + k] (int32 or int64, all
    distinct) of every pool; child j of the group continues beam parents[b, j]
    ([batch, beams], the same dtype).  The first child of a parent keeps its
    row, the others take the rows of beams without a child, which are
    overwritten with their parents' rows; no other row changes.  ``pools`` is one
    pool or a list of pools (any state dtypes and shapes, the same number of
    rows; pools that share elements are refused), all reordered alike, or none if
    one of them is refused.

    Returns the children's rows, like state_indices (in ``output_indices`` if
    given, which must not overlap the other lists).  A parent outside
    [0, beams) is none: its child takes a row that is left over, as it is; rows
    outside the pool are handed on untouched.  Both set GDN_STATUS_POOL_ROW in
    ``status`` (-1 does not: padding), a row that is named twice sets
    GDN_STATUS_POOL_DUPLICATE and is left with unspecified values.  As with
    torch's in-place operators a pool must not require a gradient (but under
    torch.no_grad()), and its autograd version advances."""
    pools = list(pools) if isinstance(pools, (list, tuple)) else [pools]
    return calls().pool_reorder(pools, state_indices, parents, output_indices, status)
