"""Python binding of the short causal convolution (include/gdn_prefill.h,
gdn_convolution*), which layers put in front of a recurrence.

Torch provides device memory and the current stream, every step of the
computation runs in the HIP kernels, and without the built library or a gfx950
device the calls raise.  Arguments are checked and marshalled by ``_calls``.
"""
from __future__ import annotations

import torch

from ._launch import calls
from .api import _QKV_DTYPES
from .recurrence import _capturing

_ACTIVATIONS = {None: False, "silu": True}


def _silu(activation):
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or \"silu\"")
    return _ACTIVATIONS[activation]


class _Convolution(torch.autograd.Function):
    """The forward call with its gradient; the arguments are the tensors that
    take one, then the others."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, silu, cu_seqlens, output_final_state):
        out, final = calls().conv_forward(x, weight, bias, silu, initial_state, output_final_state,
                                          cu_seqlens, None, None, None, None, None)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu = silu
        return (out, final) if output_final_state else out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dfinal=None):
        x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
        if _capturing(x):
            raise RuntimeError("autograd through short_convolution cannot be captured into a "
                               "graph; capture short_convolution_backward instead")
        want0 = initial_state is not None and ctx.needs_input_grad[3]
        dout = torch.zeros_like(x, memory_format=torch.contiguous_format) if dout is None \
            else dout.contiguous()
        res = calls().conv_backward(
            dout, x, weight, bias, ctx.silu, initial_state,
            None if dfinal is None else dfinal.contiguous(), cu_seqlens, want0,
            None, None, None, None, None, None)
        return (res[0], res[1].to(weight.dtype), None if bias is None else res[2].to(bias.dtype),
                res[3].to(initial_state.dtype) if want0 else None, None, None, None)


def short_convolution(x, weight, bias=None, activation=None, initial_state=None,
                      output_final_state=False, cu_seqlens=None, output=None, output_state=None,
                      state_indices=None, status=None, workspace=None):
    """Causal depthwise convolution over the last 2 to 4 tokens, on the current
    stream: output_t = act(bias + sum_j weight[:, j] x~_{t + j}) with x~ a
    sequence's state followed by its tokens.

    x [T, C] float32, bfloat16 or float16 (a token's channels are contiguous,
    tokens may be strided: a slice of a wider projection); weight [C, W], bias
    [C] float32 or x's dtype, W 2, 3 or 4; ``activation`` None or "silu".
    cu_seqlens [N+1] int32/int64 packs N sequences (None: one).  A state holds a
    sequence's last W - 1 inputs, oldest first: [N or pool, W - 1, C] in any
    state dtype, rows may be strided; with ``state_indices`` [N] sequence i
    starts from ``initial_state`` row state_indices[i] and leaves its final
    state in that row of ``output_state``, which may be ``initial_state``
    itself; rows must then be unique.  Sums are formed in float32.  No other two
    tensors of a call may overlap.

    ``workspace`` (optional uint8 device tensor) is used, if it is large
    enough, instead of the one that is kept for the current stream; only batches
    of more than 63 sequences need one, for themselves until their kernels have
    ended.

    Returns ``output`` [T, C] (rows outside every sequence are not written),
    with ``output_final_state`` also the final state.  A tensor that the call
    writes must not require a gradient (but under torch.no_grad()), and its
    autograd version advances.

    Where x, weight, bias or initial_state require a gradient (and grad mode is
    on) the call is differentiable; it then takes no output buffers,
    state_indices, status or workspace, initial_state is float32, bfloat16 or
    float16, and it cannot be captured into a graph.  There are no forward-mode
    derivatives: dual tensors are refused."""
    silu = _silu(activation)
    needs = torch.is_grad_enabled() and any(
        isinstance(t, torch.Tensor) and t.requires_grad for t in (x, weight, bias, initial_state))
    if needs:
        if (output is not None or output_state is not None or state_indices is not None
                or status is not None or workspace is not None):
            raise ValueError("a differentiable call takes no output buffers, state_indices, "
                             "status or workspace; use short_convolution_backward with "
                             "torch.no_grad()")
        if initial_state is not None and initial_state.dtype not in _QKV_DTYPES:
            raise ValueError("a differentiable call's initial_state must be float32, bfloat16 "
                             "or float16")
        if isinstance(x, torch.Tensor) and _capturing(x):
            raise RuntimeError("a differentiable short_convolution cannot be captured into a "
                               "graph; use torch.no_grad() and short_convolution_backward")
        return _Convolution.apply(x, weight, bias, initial_state, silu, cu_seqlens,
                                  bool(output_final_state))
    res = calls().conv_forward(x, weight, bias, silu, initial_state, output_final_state, cu_seqlens,
                               output, output_state, state_indices, status, workspace)
    return res if output_final_state else res[0]


def short_convolution_backward(doutput, x, weight, bias=None, activation=None, initial_state=None,
                               dfinal_state=None, cu_seqlens=None, output_dinitial_state=False,
                               dx=None, dweight=None, dbias=None, dinitial_state=None,
                               status=None, workspace=None):
    """Gradients of ``short_convolution`` on the current stream.

    doutput is the gradient of output ([T, C], x's dtype), dfinal_state that of
    the final state ([N, W - 1, C] float32, None: zero); the other arguments are
    those of the forward call (initial_state [N, W - 1, C], no pool).  Returns
    (dx, dweight, dbias), with ``output_dinitial_state`` also dinitial_state: dx
    in x's dtype, the others float32, dbias None without a bias.  Rows of dx
    outside every sequence are zero.  Results do not depend on the order in
    which the work runs.  The call itself is not differentiable: tensors that
    require a gradient are refused (but under torch.no_grad())."""
    return calls().conv_backward(doutput, x, weight, bias, _silu(activation), initial_state,
                                 dfinal_state, cu_seqlens, output_dinitial_state, dx, dweight,
                                 dbias, dinitial_state, status, workspace)


def short_convolution_decode(x, weight, bias=None, activation=None, initial_state=None,
                             output_final_state=True, output=None, output_state=None,
                             state_indices=None, status=None):
    """One decode step: token i of x [N, C] is the new token of sequence i.
    States and ``state_indices`` are those of ``short_convolution``; output may
    be x itself.  Returns ``output`` [N, C], or ``(output, final_state)``.  The
    call is not differentiable: tensors that require a gradient are refused (but
    under torch.no_grad())."""
    return calls().conv_decode(x, weight, bias, _silu(activation), initial_state,
                               output_final_state, output, output_state, state_indices, status)
