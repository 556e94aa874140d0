"""GPU tests of what the recurrence and the state-pool calls owe to autograd: writes
in place are seen by graphs that saved the tensor, and nothing is detached from a
gradient without a word."""
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    PrefillGraphs, chunk_gated_delta_rule, chunk_gated_delta_rule_noalloc,
    gated_delta_rule_decode, gated_linear_recurrence, gated_linear_recurrence_backward, gated_linear_recurrence_decode,
    state_pool_compact, state_pool_copy, state_pool_reset)
from tests import recurrence_testlib as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _rows(*r):
    return torch.tensor(r, dtype=torch.int32, device="cuda")


LENS = [10, 7]


def _writers(d, pool):
    """Calls that write a [4, 2, 32] pool in place, by name."""
    idx = _rows(0, 3)
    one = d["x"][:2]
    gate = d["g"][:2]
    other = torch.zeros_like(pool)
    return {
        "reset": lambda: state_pool_reset(pool, _rows(0)),
        "copy": lambda: state_pool_copy(pool, _rows(2), _rows(0)),
        "copy in": lambda: state_pool_copy(pool, _rows(2), _rows(0), src_pool=other),
        "compact": lambda: state_pool_compact([other, pool], _rows(3, 1)),
        "forward": lambda: gated_linear_recurrence(
            d["x"], d["g"], initial_state=pool, output_final_state=True, cu_seqlens=d["cu"],
            output_state=pool, state_indices=idx),
        "decode": lambda: gated_linear_recurrence_decode(
            one, gate, initial_state=pool, output_state=pool, state_indices=idx),
    }


@pytest.mark.parametrize("name", ["reset", "copy", "copy in", "compact", "forward", "decode"])
def test_pool_writes_are_seen_by_the_graph(name):
    """A differentiable call that starts from pool rows; the pool is written
    before the backward pass: it raises, as after torch's in-place operators."""
    d = R.make(80, LENS, 2, 32)
    pool = torch.randn((4, 2, 32), device="cuda")
    x = d["x"].clone().requires_grad_()
    out = gated_linear_recurrence(x, d["g"], initial_state=pool[:2], cu_seqlens=d["cu"])
    version = pool._version
    _writers(d, pool)[name]()
    assert pool._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_buffer_writes_are_seen_by_the_graph():
    d = R.make(81, LENS, 2, 32)
    buf = d["x"].clone()
    g = d["g"].clone().requires_grad_()
    out = gated_linear_recurrence(buf, g, cu_seqlens=d["cu"])
    gated_linear_recurrence(buf, d["g"], cu_seqlens=d["cu"], output=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    # every buffer that the calls take
    T, N = d["x"].shape[0], 2
    bufs = {k: torch.empty_like(d[v]) for k, v in
            (("dx", "x"), ("dg", "g"), ("dinitial_state", "h0"))}
    st = _rows(0)
    gated_linear_recurrence_backward(d["dy"], d["x"], d["g"], cu_seqlens=d["cu"],
                                     output_dinitial_state=True, status=st, **bufs)
    assert all(b._version == 1 for b in bufs.values()) and st._version == 1
    ren, where = _rows(0, 0), _rows(0, 0, 0, 0)
    state_pool_compact(torch.zeros((4, 8), device="cuda"), _rows(1, 2), output_indices=ren,
                       row_map=where, status=st)
    assert ren._version == where._version == 1 and st._version == 2
    out1 = torch.empty((2, 2, 32), device="cuda")
    gated_linear_recurrence_decode(d["x"][:2], d["g"][:2], output=out1, output_final_state=False,
                                   status=st)
    assert out1._version == 1 and st._version == 3
    # what is only read does not change its version
    assert d["x"]._version == d["g"]._version == d["h0"]._version == 0


def test_written_tensors_that_require_a_gradient():
    d = R.make(82, LENS, 2, 32)
    leaf = torch.randn((4, 2, 32), device="cuda", requires_grad=True)
    keep = leaf.detach().clone()
    for pool in (leaf, leaf * 1.0):
        for name, call in _writers(d, pool).items():
            if name == "forward":
                continue  # differentiable there, and then takes no output_state
            with pytest.raises(ValueError):
                call()
        with pytest.raises(ValueError):
            gated_linear_recurrence(d["x"], d["g"], output=torch.empty_like(d["x"],
                                                                            requires_grad=True))
    assert torch.equal(leaf.detach(), keep)
    with torch.no_grad():
        state_pool_reset(leaf, _rows(1))
    keep[1] = 0
    assert torch.equal(leaf.detach(), keep)


def test_inference_tensors():
    d = R.make(83, LENS, 2, 32)
    with torch.inference_mode():
        pool = torch.randn((4, 2, 32), device="cuda")
        state_pool_reset(pool, _rows(1))
        assert (pool[1] == 0).all()
        gated_linear_recurrence_decode(d["x"][:2], d["g"][:2], initial_state=pool,
                                       output_state=pool, state_indices=_rows(0, 3))
    state_pool_reset(pool, _rows(2))
    assert (pool[2] == 0).all()


def test_calls_that_are_not_differentiable():
    """Tensors that require a gradient are refused where the result would be
    detached from them, and taken under no_grad."""
    d = R.make(84, LENS, 2, 32)
    need = lambda t: t.clone().requires_grad_()  # noqa: E731
    pool = torch.zeros((4, 2, 32), device="cuda")
    x, g, one, gate, h0 = d["x"], d["g"], d["x"][:2], d["g"][:2], d["h0"]
    kw = dict(cu_seqlens=d["cu"])
    calls = [
        lambda t: gated_linear_recurrence_decode(t(one), gate),
        lambda t: gated_linear_recurrence_decode(one, t(gate)),
        lambda t: gated_linear_recurrence_decode(one, gate, initial_state=t(h0)),
        lambda t: state_pool_copy(pool, _rows(0), _rows(0), src_pool=t(pool)),
        lambda t: gated_linear_recurrence_backward(t(d["dy"]), x, g, **kw),
        lambda t: gated_linear_recurrence_backward(d["dy"], t(x), g, **kw),
        lambda t: gated_linear_recurrence_backward(d["dy"], x, t(g), **kw),
        lambda t: gated_linear_recurrence_backward(d["dy"], x, g, initial_state=t(h0), **kw),
        lambda t: gated_linear_recurrence_backward(d["dy"], x, g, dfinal_state=t(d["dfinal"]),
                                                   **kw),
        lambda t: gated_linear_recurrence_backward(
            d["dy"], x, g, chunk_states=t(torch.zeros((1, 2, 32), device="cuda")), **kw),
    ]
    for call in calls:
        call(lambda t: t)
        with pytest.raises(ValueError):
            call(need)
        with torch.no_grad():
            call(need)


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as fwAD
    d = R.make(85, LENS, 2, 32)
    pool = torch.zeros((4, 2, 32), device="cuda")
    with fwAD.dual_level():
        dual = lambda t: fwAD.make_dual(t.clone(), torch.ones_like(t))  # noqa: E731
        calls = [
            lambda t: gated_linear_recurrence(t(d["x"]), d["g"]),
            lambda t: gated_linear_recurrence(d["x"], t(d["g"])),
            lambda t: gated_linear_recurrence(d["x"], d["g"], initial_state=t(d["h0"]),
                                              cu_seqlens=d["cu"]),
            lambda t: gated_linear_recurrence_decode(t(d["x"]), d["g"]),
            lambda t: state_pool_reset(t(pool), _rows(0)),
            lambda t: state_pool_copy(pool, _rows(0), _rows(0), src_pool=t(pool)),
        ]
        for call in calls:
            call(lambda t: t)
            for grad in (torch.enable_grad(), torch.no_grad()):
                with grad, pytest.raises(ValueError):
                    call(dual)
        # a tensor that requires a gradient and has a tangent
        with pytest.raises((RuntimeError, ValueError)):
            gated_linear_recurrence(fwAD.make_dual(d["x"].clone().requires_grad_(),
                                                   torch.ones_like(d["x"])), d["g"])


def test_flags_without_a_truth_value():
    """The exception of the flag itself, before anything is launched."""
    d = R.make(86, LENS, 2, 32)
    both = torch.tensor([True, False])
    out = torch.full_like(d["x"], 7.0)
    for kw in (dict(output_final_state=both), dict(return_chunk_states=both)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            gated_linear_recurrence(d["x"], d["g"], cu_seqlens=d["cu"], output=out, **kw)
    with pytest.raises(RuntimeError, match="ambiguous"):
        gated_linear_recurrence_backward(d["dy"], d["x"], d["g"], output_dinitial_state=both,
                                         dx=out)
    with pytest.raises(RuntimeError, match="ambiguous"):
        gated_linear_recurrence_decode(d["x"], d["g"], output=out, output_final_state=both)
    torch.cuda.synchronize()
    assert (out == 7).all()


@pytest.mark.parametrize("name", ["prefill", "noalloc", "graphs", "decode"])
def test_writes_of_the_delta_rule_are_seen_by_the_graph(name):
    """Its output buffer is the recurrence's x, its pool holds the recurrence's
    initial states too: written again before the backward pass, both raise."""
    H, D = 2, 32
    gen = torch.Generator(device="cuda").manual_seed(87)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    T = 3 if name == "decode" else 20
    q, k, v = rand(T, H, D), rand(T, H, D), rand(T, H, D)
    buf, pool = torch.zeros((T, H, D), device="cuda"), rand(4, H, D, D)
    rows = _rows(0, 3, 1) if name == "decode" else _rows(2)
    st = _rows(0)
    call = {"prefill": chunk_gated_delta_rule, "noalloc": chunk_gated_delta_rule_noalloc,
            "graphs": PrefillGraphs(), "decode": gated_delta_rule_decode}[name]

    def step():
        call(q, k, v, initial_state=pool, output_final_state=True, output=buf, output_state=pool,
             state_indices=rows, use_qk_l2norm_in_kernel=True, status=st)

    step()
    gate = torch.rand((T, H, D), generator=gen, device="cuda").requires_grad_()
    start = pool.view(4 * D, H, D)[:1]
    for kw in (dict(), dict(initial_state=start)):
        x = buf if not kw else rand(T, H, D)
        gated_linear_recurrence(x, gate, **kw).sum().backward()
        out = gated_linear_recurrence(x, gate, **kw)
        versions = buf._version, pool._version, st._version
        step()
        assert all(a > b for a, b in zip((buf._version, pool._version, st._version), versions))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()
    assert q._version == 0
    with torch.inference_mode():
        o = chunk_gated_delta_rule(q, k, v)
    assert o.is_inference()


def test_autograd_without_tokens_or_sequences():
    """The incoming gradients of sums are expanded, and an empty tensor stays so
    when it is made contiguous."""
    x = torch.zeros((0, 2, 32), device="cuda", requires_grad=True)
    g = torch.zeros((0, 2, 32), device="cuda")
    h0 = torch.randn((3, 2, 32), device="cuda", requires_grad=True)
    out, fin = gated_linear_recurrence(x, g, initial_state=h0, output_final_state=True,
                                       cu_seqlens=_rows(0, 0, 0, 0))
    (out.sum() + 2 * fin.sum()).backward()
    assert (h0.grad == 2).all() and x.grad.shape == x.shape
    x = torch.randn((5, 2, 32), device="cuda", requires_grad=True)
    h0 = torch.zeros((1, 2, 1), device="cuda", requires_grad=True)
    out, fin = gated_linear_recurrence(x, x.detach().sigmoid(), cu_seqlens=_rows(0),
                                       initial_state=h0.expand(1, 2, 32)[:0],
                                       output_final_state=True)
    fin.sum().backward()
    assert (x.grad == 0).all() and (h0.grad == 0).all() and fin.shape == (0, 2, 32)
