"""Python binding of the gated linear recurrence (include/gdn_prefill.h,
gdn_recurrence*): h_t = g_t * h_{t-1} + x_t over packed sequences.

Argument marshalling only, in the manner of ``api``: torch provides device
memory and the current stream, every step of the computation runs in the HIP
kernels, and without the built library or a gfx950 device the calls raise.
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import _launch
from . import _native as nat
from ._launch import Blocks, meta
from .api import (_QKV_DTYPES, _STATE_DTYPES, _check_dev, _index, state_tensor,
                  workspace_tensor)


def _token_stride(name, t, inner):
    """Token stride in elements of a [T, ...] tensor whose tokens each hold
    ``inner`` contiguous values; anything else raises."""
    want = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and st != want:
            raise ValueError("%s: a token's values must be contiguous" % name)
        want *= n
    if t.shape[0] <= 1:
        return inner
    if t.stride(0) < inner:
        raise ValueError("%s must not overlap itself (token stride %d < %d)"
                         % (name, t.stride(0), inner))
    return int(t.stride(0))


def _rec_state(name, t, rows, H, D, written):
    """Checks a [rows, H, D] state tensor; returns it and its row stride."""
    if t.dtype not in _STATE_DTYPES:
        raise ValueError("unsupported %s dtype" % name)
    if tuple(t.shape) != (rows, H, D):
        raise ValueError("%s must be [%d, %d, %d]" % (name, rows, H, D))
    t = state_tensor(name, t, written)
    return t, _token_stride(name, t, H * D)


def _contiguous(name, t, shape, dtype):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s %s" % (name, list(shape), dtype))


def _base_params(x, g, cu_seqlens, decode, tensors):
    """Shapes, types and devices shared by the three calls."""
    if not (isinstance(x, torch.Tensor) and isinstance(g, torch.Tensor)):
        raise ValueError("x and g must be tensors")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    for name, t in tensors:
        _check_dev(name, t, x.device)
    if x.dim() != 3:
        raise ValueError("x must be [total_seq_len, heads, head_size]")
    if x.dtype not in _QKV_DTYPES:
        raise ValueError("x must be float32, bfloat16 or float16")
    if g.dtype not in (torch.float32, x.dtype):
        raise ValueError("g must be float32 or x's dtype")
    T, H, D = x.shape
    per_head = g.dim() == 2
    if tuple(g.shape) != ((T, H) if per_head else (T, H, D)):
        raise ValueError("g must be [%d, %d, %d] or [%d, %d]" % (T, H, D, T, H))
    if H < 1 or D < 1:
        raise ValueError("x needs at least one head and one channel")
    p = nat.RecurrenceParams()
    p.total_tokens, p.num_heads, p.head_size = T, H, D
    p.x_dtype, p.g_dtype = _QKV_DTYPES[x.dtype], _QKV_DTYPES[g.dtype]
    p.g_per_head = 1 if per_head else 0
    p.x_stride = _token_stride("x", x, H * D)
    p.g_stride = _token_stride("g", g, H if per_head else H * D)
    if decode:
        p.num_seqs = T
    elif cu_seqlens is not None:
        p.cu_seqlens_type = _index("cu_seqlens", cu_seqlens)
        if cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must hold at least one offset")
        p.num_seqs = cu_seqlens.numel() - 1
    else:
        p.num_seqs = 1
    return p


def _status(status):
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status must be an int32 tensor")


def _states(p, x, initial_state, output_final_state, output_state, state_indices):
    """Checks and fills in the initial, final and pool states of a forward or
    decode call; returns (initial_state to read, rows of the final state)."""
    N, (_, H, D) = p.num_seqs, x.shape
    rows = N
    if state_indices is not None:
        p.state_indices_type = _index("state_indices", state_indices)
        if state_indices.numel() != N:
            raise ValueError("state_indices must hold %d rows" % N)
        pool = output_state if output_state is not None else initial_state
        if pool is None:
            raise ValueError("state_indices needs a state pool")
        p.pool_size = rows = pool.shape[0]
    if initial_state is not None:
        initial_state, stride = _rec_state("initial_state", initial_state, rows, H, D, False)
        p.initial_state_dtype = _STATE_DTYPES[initial_state.dtype]
        p.initial_state_stride = stride
    if output_final_state:
        p.output_final_state = 1
        if output_state is None:
            if state_indices is not None:
                raise ValueError("output_state (the pool) is required with state_indices")
            p.output_state_dtype, p.output_state_stride = nat.GDN_F32, H * D
        else:
            output_state, stride = _rec_state("output_state", output_state, rows, H, D, True)
            p.output_state_dtype = _STATE_DTYPES[output_state.dtype]
            p.output_state_stride = stride
    return initial_state


_forward_blocks = Blocks(nat.RecurrenceParams)
_backward_blocks = Blocks(nat.RecurrenceParams)
_decode_blocks = Blocks(nat.RecurrenceParams)


def _memory(p, device, need, workspace):
    """Puts the workspace of a scan into its parameter block; returns it."""
    if workspace is not None:
        workspace = workspace_tensor(workspace, device, need)
    elif need > 0:
        if torch.cuda.current_device() == device.index:
            workspace = _launch.workspace(device, need)
        else:
            with torch.cuda.device(device):
                workspace = _launch.workspace(device, need)
    else:
        return None
    p.workspace, p.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return workspace


def _new_like(x):
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _forward(x, g, initial_state, output_final_state, cu_seqlens, output, output_state,
             state_indices, return_chunk_states, status, workspace):
    """Returns (output, final state or None, chunk states or None)."""
    try:
        key = (x.shape, x.stride(), x.dtype, x.device, g.shape, g.stride(), g.dtype, g.device,
               meta(initial_state), bool(output_final_state), meta(cu_seqlens), meta(output),
               meta(output_state), meta(state_indices), meta(status), bool(return_chunk_states))
        hit = _forward_blocks.get(key)
    except AttributeError:
        raise ValueError("x, g and the optional arguments must be tensors") from None
    if hit is None:
        p = _base_params(x, g, cu_seqlens, False, (
            ("g", g), ("initial_state", initial_state), ("cu_seqlens", cu_seqlens),
            ("output", output), ("output_state", output_state), ("state_indices", state_indices),
            ("status", status)))
        if output is not None:
            _contiguous("output", output, x.shape, x.dtype)
        _status(status)
        used = _states(p, x, initial_state, output_final_state, output_state, state_indices)
        need = _workspace_size(p, cu_seqlens, False)
        if used is initial_state:
            _forward_blocks.keep(key, p, need)
        initial_state = used
    else:
        p, need = hit
    if output is None:
        output = _new_like(x)
    p.x, p.g, p.output = x.data_ptr(), g.data_ptr(), output.data_ptr()
    if cu_seqlens is not None:
        p.cu_seqlens = cu_seqlens.data_ptr()
    if initial_state is not None:
        p.initial_state = initial_state.data_ptr()
    if output_final_state:
        if output_state is None:
            output_state = torch.empty((p.num_seqs,) + x.shape[1:], dtype=torch.float32,
                                       device=x.device)
        p.output_state = output_state.data_ptr()
    if state_indices is not None:
        p.state_indices = state_indices.data_ptr()
    kept = None
    if return_chunk_states:
        kept = torch.empty(_chunk_shape(x), dtype=torch.float32, device=x.device)
        p.chunk_states = kept.data_ptr()
    if status is not None:
        p.status = status.data_ptr()
    memory = _memory(p, x.device, need, workspace)
    _launch.call(nat.lib().gdn_recurrence, x.device, byref(p))
    del memory
    return output, (output_state if output_final_state else None), kept


def _workspace_size(p, cu_seqlens, backward):
    """Workspace of a scan whose block has no addresses yet (the library looks
    only at which of them are there)."""
    p.cu_seqlens = None if cu_seqlens is None else cu_seqlens.data_ptr()
    need = int(nat.lib().gdn_recurrence_workspace_size(byref(p), int(backward)))
    p.cu_seqlens = None
    return need


def _chunk_shape(x):
    return (-(-x.shape[0] // nat.RECURRENCE_CHUNK), x.shape[1], x.shape[2])


class _Recurrence(torch.autograd.Function):
    """The forward call with its gradient; the arguments are the tensors that
    take one, then cu_seqlens and whether the final state is returned."""

    @staticmethod
    def forward(ctx, x, g, initial_state, cu_seqlens, output_final_state):
        out, final, kept = _forward(x, g, initial_state, output_final_state, cu_seqlens, None,
                                    None, None, True, None, None)
        ctx.save_for_backward(x, g, initial_state, cu_seqlens, kept)
        ctx.with_final = output_final_state
        return (out, final) if output_final_state else out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dfinal=None):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("autograd through gated_linear_recurrence cannot be captured into "
                               "a graph; capture gated_linear_recurrence_backward instead")
        x, g, initial_state, cu_seqlens, kept = ctx.saved_tensors
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
    ``output_state``, which may be ``initial_state`` itself.  h is fp32
    throughout.

    Returns ``output`` [T, H, D] (rows outside every sequence are not
    written), then the final state with ``output_final_state``, then with
    ``return_chunk_states`` the float32 states that
    ``gated_linear_recurrence_backward`` starts from.

    Where x, g or initial_state require a gradient (and grad mode is on) the
    call is differentiable; it then takes no output buffers, state_indices,
    status or workspace, initial_state is float32, bfloat16 or float16, and it
    cannot be captured into a graph."""
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
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a differentiable gated_linear_recurrence cannot be captured into "
                               "a graph; use torch.no_grad() and "
                               "gated_linear_recurrence_backward")
        return _Recurrence.apply(x, g, initial_state, cu_seqlens, bool(output_final_state))
    res = _forward(x, g, initial_state, output_final_state, cu_seqlens, output, output_state,
                   state_indices, return_chunk_states, status, workspace)
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
    not depend on the order in which the work runs."""
    try:
        key = (x.shape, x.stride(), x.dtype, x.device, g.shape, g.stride(), g.dtype, g.device,
               doutput.shape, doutput.stride(), doutput.dtype, doutput.device,
               meta(initial_state), meta(dfinal_state), meta(cu_seqlens), meta(chunk_states),
               bool(output_dinitial_state), meta(dx), meta(dg), meta(dinitial_state),
               meta(status))
        hit = _backward_blocks.get(key)
    except AttributeError:
        raise ValueError("doutput, x, g and the optional arguments must be tensors") from None
    if hit is None:
        p = _base_params(x, g, cu_seqlens, False, (
            ("g", g), ("doutput", doutput), ("initial_state", initial_state),
            ("dfinal_state", dfinal_state), ("cu_seqlens", cu_seqlens),
            ("chunk_states", chunk_states), ("dx", dx), ("dg", dg),
            ("dinitial_state", dinitial_state), ("status", status)))
        N, (_, H, D) = p.num_seqs, x.shape
        if doutput.dtype != x.dtype or doutput.shape != x.shape:
            raise ValueError("doutput must have x's shape and dtype")
        p.doutput_stride = _token_stride("doutput", doutput, H * D)
        used = initial_state
        if initial_state is not None:
            used, stride = _rec_state("initial_state", initial_state, N, H, D, False)
            p.initial_state_dtype = _STATE_DTYPES[used.dtype]
            p.initial_state_stride = stride
        for name, t, shape, dtype in (
                ("dfinal_state", dfinal_state, (N, H, D), torch.float32),
                ("chunk_states", chunk_states, _chunk_shape(x), torch.float32),
                ("dx", dx, x.shape, x.dtype), ("dg", dg, g.shape, g.dtype),
                ("dinitial_state", dinitial_state, (N, H, D), torch.float32)):
            if t is not None:
                _contiguous(name, t, shape, dtype)
        _status(status)
        p.chunk_states = None if chunk_states is None else chunk_states.data_ptr()
        need = _workspace_size(p, cu_seqlens, True)
        p.chunk_states = None
        if used is initial_state:
            _backward_blocks.keep(key, p, need)
        initial_state = used
    else:
        p, need = hit
    if dx is None:
        dx = _new_like(x)
    if dg is None:
        dg = _new_like(g)
    p.x, p.g, p.doutput = x.data_ptr(), g.data_ptr(), doutput.data_ptr()
    p.dx, p.dg = dx.data_ptr(), dg.data_ptr()
    if cu_seqlens is not None:
        p.cu_seqlens = cu_seqlens.data_ptr()
    if initial_state is not None:
        p.initial_state = initial_state.data_ptr()
    if dfinal_state is not None:
        p.dfinal_state = dfinal_state.data_ptr()
    if chunk_states is not None:
        p.chunk_states = chunk_states.data_ptr()
    if output_dinitial_state:
        if dinitial_state is None:
            dinitial_state = torch.empty((p.num_seqs,) + x.shape[1:], dtype=torch.float32,
                                         device=x.device)
        p.dinitial_state = dinitial_state.data_ptr()
    if status is not None:
        p.status = status.data_ptr()
    memory = _memory(p, x.device, need, workspace)
    _launch.call(nat.lib().gdn_recurrence_backward, x.device, byref(p))
    del memory
    return (dx, dg, dinitial_state) if output_dinitial_state else (dx, dg)


def gated_linear_recurrence_decode(x, g, initial_state=None, output_final_state=True, output=None,
                                   output_state=None, state_indices=None, status=None):
    """One decode step: token i of x, g [N, ...] is the new token of sequence
    i.  States and ``state_indices`` are those of ``gated_linear_recurrence``.
    Returns ``output`` [N, H, D], or ``(output, final_state)``."""
    try:
        key = (x.shape, x.stride(), x.dtype, x.device, g.shape, g.stride(), g.dtype, g.device,
               meta(initial_state), bool(output_final_state), meta(output), meta(output_state),
               meta(state_indices), meta(status))
        hit = _decode_blocks.get(key)
    except AttributeError:
        raise ValueError("x, g and the optional arguments must be tensors") from None
    if hit is None:
        p = _base_params(x, g, None, True, (
            ("g", g), ("initial_state", initial_state), ("output", output),
            ("output_state", output_state), ("state_indices", state_indices),
            ("status", status)))
        if output is not None:
            _contiguous("output", output, x.shape, x.dtype)
        _status(status)
        used = _states(p, x, initial_state, output_final_state, output_state, state_indices)
        if used is initial_state:
            _decode_blocks.keep(key, p)
        initial_state = used
    else:
        p = hit[0]
    if output is None:
        output = _new_like(x)
    p.x, p.g, p.output = x.data_ptr(), g.data_ptr(), output.data_ptr()
    if initial_state is not None:
        p.initial_state = initial_state.data_ptr()
    if output_final_state:
        if output_state is None:
            output_state = torch.empty((p.num_seqs,) + x.shape[1:], dtype=torch.float32,
                                       device=x.device)
        p.output_state = output_state.data_ptr()
    if state_indices is not None:
        p.state_indices = state_indices.data_ptr()
    if status is not None:
        p.status = status.data_ptr()
    _launch.call(nat.lib().gdn_recurrence_decode, x.device, byref(p))
    return (output, output_state) if output_final_state else output
