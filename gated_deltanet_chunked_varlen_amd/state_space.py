"""Python binding of the selective state space scan (include/gdn_prefill.h,
gdn_scan*).

Torch provides device memory and the current stream, every step of the
computation runs in the HIP kernels, and without the built library or a gfx950
device the calls raise.  Arguments are checked and marshalled by ``_calls``.
"""
from __future__ import annotations

import torch

from ._launch import calls
from .api import _QKV_DTYPES
from .recurrence import _capturing


class _Scan(torch.autograd.Function):
    """The forward call with its gradient; the arguments are the tensors that
    take one, then the others."""

    @staticmethod
    def forward(ctx, x, delta, A, B, C, D, z, delta_bias, initial_state, delta_softplus,
                cu_seqlens, output_final_state):
        out, final, kept = calls().scan_forward(
            x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, output_final_state,
            cu_seqlens, None, None, None, True, None, None)
        ctx.save_for_backward(x, delta, A, B, C, D, z, delta_bias, initial_state, cu_seqlens, kept)
        ctx.delta_softplus = delta_softplus
        return (out, final) if output_final_state else out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dfinal=None):
        *args, initial_state, cu_seqlens, kept = ctx.saved_tensors
        x = args[0]
        if _capturing(x):
            raise RuntimeError("autograd through selective_scan cannot be captured into a graph; "
                               "capture selective_scan_backward instead")
        want0 = initial_state is not None and ctx.needs_input_grad[8]
        dout = torch.zeros_like(x, memory_format=torch.contiguous_format) if dout is None \
            else dout.contiguous()
        res = calls().scan_backward(
            dout, *args, ctx.delta_softplus, None if initial_state is None else initial_state.float(),
            None if dfinal is None else dfinal.contiguous(), cu_seqlens, kept, want0, None, None)
        d0 = res[8].to(initial_state.dtype) if want0 else None
        return (*res[:8], d0, None, None, None)


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False,
                   initial_state=None, output_final_state=False, cu_seqlens=None, output=None,
                   output_state=None, state_indices=None, return_chunk_states=False, status=None,
                   workspace=None):
    """Selective state space scan on the current stream: with the step size
    d_t = delta_t + delta_bias (``delta_softplus``: log(1 + e^ of it)), for
    every channel and each of its states

        h_t = exp(d_t A) h_{t-1} + d_t B_t x_t
        y_t = sum over states C_t h_t + D x_t,   output_t = y_t silu(z_t)

    (without z, output_t = y_t).  x, delta, z [T, channels] float32, bfloat16 or
    float16, B and C [T, groups, states] of x's dtype (channel c belongs to group
    c // (channels / groups)), A [channels, states], D and delta_bias [channels]
    float32; 1 to 64 states.  A token's values are contiguous; tokens of x,
    delta, z, B and C may be strided.  cu_seqlens [N+1] int32/int64 packs N
    sequences (None: one).  States are [N or pool, channels, states] in any
    state dtype, rows may be strided; with ``state_indices`` [N] sequence i
    starts from ``initial_state`` row state_indices[i] and leaves its final
    state in that row of ``output_state``, which may be ``initial_state`` itself;
    rows must then be unique.  h is float32 throughout.  The products exp(A sum d)
    over 256 consecutive tokens must stay finite: they do for A <= 0 and d >= 0.
    No other two tensors of a call may overlap.

    ``workspace`` (optional uint8 device tensor) is used, if it is large
    enough, instead of the one that is kept for the current stream.  A call
    needs it for itself until its kernels have ended.

    Returns ``output`` [T, channels] (rows outside every sequence are not
    written), then the final state with ``output_final_state``, then with
    ``return_chunk_states`` the float32 states that ``selective_scan_backward``
    starts from.  A tensor that the call writes must not require a gradient (but
    under torch.no_grad()), and its autograd version advances.

    Where an input requires a gradient (and grad mode is on) the call is
    differentiable; it then takes no output buffers, state_indices, status or
    workspace, initial_state is float32, bfloat16 or float16, and it cannot be
    captured into a graph.  There are no forward-mode derivatives: dual tensors
    are refused."""
    needs = torch.is_grad_enabled() and any(
        isinstance(t, torch.Tensor) and t.requires_grad
        for t in (x, delta, A, B, C, D, z, delta_bias, initial_state))
    if needs:
        if (output is not None or output_state is not None or state_indices is not None
                or return_chunk_states or status is not None or workspace is not None):
            raise ValueError("a differentiable call takes no output buffers, state_indices, "
                             "status or workspace and returns no chunk states; use "
                             "selective_scan_backward with torch.no_grad()")
        if initial_state is not None and initial_state.dtype not in _QKV_DTYPES:
            raise ValueError("a differentiable call's initial_state must be float32, bfloat16 "
                             "or float16")
        if isinstance(x, torch.Tensor) and _capturing(x):
            raise RuntimeError("a differentiable selective_scan cannot be captured into a graph; "
                               "use torch.no_grad() and selective_scan_backward")
        return _Scan.apply(x, delta, A, B, C, D, z, delta_bias, initial_state,
                           bool(delta_softplus), cu_seqlens, bool(output_final_state))
    res = calls().scan_forward(x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state,
                               output_final_state, cu_seqlens, output, output_state, state_indices,
                               return_chunk_states, status, workspace)
    if output_final_state:
        return res if return_chunk_states else res[:2]
    return (res[0], res[2]) if return_chunk_states else res[0]


def selective_scan_backward(doutput, x, delta, A, B, C, D=None, z=None, delta_bias=None,
                            delta_softplus=False, initial_state=None, dfinal_state=None,
                            cu_seqlens=None, chunk_states=None, output_dinitial_state=False,
                            status=None, workspace=None):
    """Gradients of ``selective_scan`` on the current stream.

    doutput is the gradient of output ([T, channels], x's dtype), dfinal_state
    that of the final state ([N, channels, states] float32, None: zero); the
    other inputs are those of the forward call (initial_state float32
    [N, channels, states], no pool), and chunk_states what it returned (None:
    formed again, one more pass).  Returns (dx, ddelta, dA, dB, dC, dD, dz,
    ddelta_bias), with ``output_dinitial_state`` also dinitial_state: shapes and
    dtypes of the inputs, None for an input that was not given.  Rows outside
    every sequence are zero.  Results do not depend on the order in which the
    work runs.  The call itself is not differentiable: tensors that require a
    gradient are refused (but under torch.no_grad())."""
    return calls().scan_backward(doutput, x, delta, A, B, C, D, z, delta_bias, delta_softplus,
                                 initial_state, dfinal_state, cu_seqlens, chunk_states,
                                 output_dinitial_state, status, workspace)


def selective_scan_decode(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False,
                          initial_state=None, output_final_state=True, output=None,
                          output_state=None, state_indices=None, status=None):
    """One decode step: token i of x, delta, z [N, channels], B and C [N, groups,
    states] is the new token of sequence i.  States and ``state_indices`` are
    those of ``selective_scan``.  Returns ``output`` [N, channels], or
    ``(output, final_state)``.  The call is not differentiable: tensors that
    require a gradient are refused (but under torch.no_grad())."""
    return calls().scan_decode(x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state,
                               output_final_state, output, output_state, state_indices, status)
