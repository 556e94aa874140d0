"""Python binding of the gated linear recurrence (include/gdn_prefill.h,
gdn_recurrence*): h_t = g_t * h_{t-1} + x_t over packed sequences.

Torch provides device memory and the current stream, every step of the
computation runs in the HIP kernels, and without the built library or a gfx950
device the calls raise.  Arguments are checked and marshalled by ``_calls``.
"""
from __future__ import annotations

import torch

from ._launch import calls
from .api import _QKV_DTYPES


def _capturing(t):
    """Whether the current stream of a device tensor's own device is being
    captured (another device may be the current one)."""
    if not t.is_cuda:
        return False
    with torch.cuda.device(t.device):
        return torch.cuda.is_current_stream_capturing()


class _Recurrence(torch.autograd.Function):
    """The forward call with its gradient; the arguments are the tensors that
    take one, then cu_seqlens and whether the final state is returned."""

    @staticmethod
    def forward(ctx, x, g, initial_state, cu_seqlens, output_final_state):
        out, final, kept = calls().rec_forward(x, g, initial_state, output_final_state, cu_seqlens,
                                               None, None, None, True, None, None)
        ctx.save_for_backward(x, g, initial_state, cu_seqlens, kept)
        ctx.with_final = output_final_state
        return (out, final) if output_final_state else out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dfinal=None):
        x, g, initial_state, cu_seqlens, kept = ctx.saved_tensors
        if _capturing(x):
            raise RuntimeError("autograd through gated_linear_recurrence cannot be captured into "
                               "a graph; capture gated_linear_recurrence_backward instead")
        want0 = initial_state is not None and ctx.needs_input_grad[2]
        dout = torch.zeros_like(x, memory_format=torch.contiguous_format) if dout is None \
            else dout.contiguous()
        res = gated_linear_recurrence_backward(
            dout, x, g, initial_state=initial_state,
            dfinal_state=None if dfinal is None else dfinal.contiguous(), cu_seqlens=cu_seqlens,
            chunk_states=kept, output_dinitial_state=want0)
        d0 = res[2].to(initial_state.dtype) if want0 else None
        return res[0], res[1], d0, None, None


def gated_linear_recurrence(x, g, initial_state=None, output_final_state=False, cu_seqlens=None,
                            output=None, output_state=None, state_indices=None,
                            return_chunk_states=False, status=None, workspace=None):
    """Gated linear recurrence h_t = g_t * h_{t-1} + x_t on the current stream.

    x [T, H, D] float32, bfloat16 or float16; g, the forget gate itself in
    [0, 1], float32 or x's dtype: [T, H, D], or [T, H] for one gate per head
    (head size 32, 64 or 128).  A token's values are contiguous; tokens may be
    strided.  cu_seqlens [N+1] int32/int64 packs N sequences (None: one).
    States are [N or pool, H, D] in any state dtype, rows may be strided; with
    ``state_indices`` [N] sequence i starts from ``initial_state`` row
    state_indices[i] and leaves its final state in that row of
    ``output_state``, which may be ``initial_state`` itself; rows must then be
    unique (sequences may share a start row where no final state is written).
    h is fp32 throughout.  ``output`` may be x itself; no other two tensors of
    a call may overlap.

    ``workspace`` (optional uint8 device tensor) is used, if it is large
    enough, instead of the one that is kept for the current stream.  A call
    needs it for itself until its kernels have ended: calls on two streams at
    once (or two captured graphs that run at once) with one workspace give
    wrong values.

    Returns ``output`` [T, H, D] (rows outside every sequence are not
    written), then the final state with ``output_final_state``, then with
    ``return_chunk_states`` the float32 states that
    ``gated_linear_recurrence_backward`` starts from.

    A tensor that the call writes must not require a gradient (but under
    torch.no_grad()), and its autograd version advances.

    Where x, g or initial_state require a gradient (and grad mode is on) the
    call is differentiable; it then takes no output buffers, state_indices,
    status or workspace, initial_state is float32, bfloat16 or float16, and it
    cannot be captured into a graph.  There are no forward-mode derivatives:
    dual tensors are refused."""
    needs = torch.is_grad_enabled() and any(
        isinstance(t, torch.Tensor) and t.requires_grad for t in (x, g, initial_state))
    if needs:
        if (output is not None or output_state is not None or state_indices is not None
                or return_chunk_states or status is not None or workspace is not None):
            raise ValueError("a differentiable call takes no output buffers, state_indices, "
                             "status or workspace and returns no chunk states; use "
                             "gated_linear_recurrence_backward with torch.no_grad()")
        if initial_state is not None and initial_state.dtype not in _QKV_DTYPES:
            raise ValueError("a differentiable call's initial_state must be float32, bfloat16 "
                             "or float16")
        if isinstance(x, torch.Tensor) and _capturing(x):
            raise RuntimeError("a differentiable gated_linear_recurrence cannot be captured into "
                               "a graph; use torch.no_grad() and "
                               "gated_linear_recurrence_backward")
        return _Recurrence.apply(x, g, initial_state, cu_seqlens, bool(output_final_state))
    res = calls().rec_forward(x, g, initial_state, output_final_state, cu_seqlens, output,
                              output_state, state_indices, return_chunk_states, status, workspace)
    if output_final_state:
        return res if return_chunk_states else res[:2]
    return (res[0], res[2]) if return_chunk_states else res[0]


def gated_linear_recurrence_backward(doutput, x, g, initial_state=None, dfinal_state=None,
                                     cu_seqlens=None, chunk_states=None,
                                     output_dinitial_state=False, dx=None, dg=None,
                                     dinitial_state=None, status=None, workspace=None):
    """Gradients of ``gated_linear_recurrence`` on the current stream.

    doutput is the gradient of output ([T, H, D], x's dtype), dfinal_state that
    of the final state ([N, H, D] float32, None: zero); x, g, initial_state
    ([N, H, D], no pool) and cu_seqlens are those of the forward call, and
    chunk_states what it returned (None: formed again, one more pass over x
    and g).  Returns (dx, dg), or (dx, dg, dinitial_state) with
    ``output_dinitial_state``: x's and g's shapes and dtypes, float32
    [N, H, D].  Rows of dx and dg outside every sequence are zero.  Results do
    not depend on the order in which the work runs.  No two tensors of a call
    may overlap, and ``workspace`` is used as in the forward call.  The call
    itself is not differentiable: tensors that require a gradient are refused
    (but under torch.no_grad())."""
    return calls().rec_backward(doutput, x, g, initial_state, dfinal_state, cu_seqlens,
                                chunk_states, output_dinitial_state, dx, dg, dinitial_state,
                                status, workspace)


def gated_linear_recurrence_decode(x, g, initial_state=None, output_final_state=True, output=None,
                                   output_state=None, state_indices=None, status=None):
    """One decode step: token i of x, g [N, ...] is the new token of sequence
    i.  States and ``state_indices`` are those of ``gated_linear_recurrence``.
    Returns ``output`` [N, H, D], or ``(output, final_state)``.  The call is
    not differentiable: tensors that require a gradient are refused (but under
    torch.no_grad())."""
    return calls().rec_decode(x, g, initial_state, output_final_state, output, output_state,
                              state_indices, status)
