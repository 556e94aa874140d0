"""GPU tests of the operators as a serving loop or a training step uses them: a
convolution in front of the gated delta rule, beam search over the pools of
both, graphs, streams and threads."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gated_deltanet_chunked_varlen_amd as gdn  # noqa: E402
from tests import layers_testlib as L  # noqa: E402
from tests.recurrence_testlib import f64  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


class Model:
    """One layer: convolution, then the gated delta rule (or the selective scan),
    with random weights; a head over a small vocabulary."""

    def __init__(self, kind, H=2, D=32, V=50):
        gen = torch.Generator().manual_seed(5)
        rnd = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
        self.kind, self.H, self.D, self.V = kind, H, D, V
        self.C = 3 * H * D
        self.emb, self.w = rnd(V, self.C), 0.5 * rnd(self.C, 4)
        self.g = 0.5 + 0.5 * torch.rand((V, H), generator=gen).cuda()
        self.beta = torch.rand((V, H), generator=gen).cuda()
        self.A, self.B, self.Cm = -torch.exp(rnd(self.C, 8)), rnd(V, 1, 8), rnd(V, 1, 8)
        self.head = rnd(H * D if kind == "delta" else self.C, V)

    def pools(self, rows):
        conv = torch.zeros((rows, 3, self.C), device="cuda")
        if self.kind == "delta":
            return [conv, torch.zeros((rows, self.H, self.D, self.D), device="cuda")]
        return [conv, torch.zeros((rows, self.C, 8), device="cuda")]

    def run(self, tokens, pools, idx, cu=None):
        """Outputs of the tokens; the sequences' states in rows idx of the pools."""
        x, (conv, state) = self.emb[tokens], pools
        at = dict(initial_state=conv, output_state=conv, state_indices=idx)
        if cu is None:
            y, _ = gdn.short_convolution_decode(x, self.w, activation="silu", **at)
        else:
            y, _ = gdn.short_convolution(x, self.w, activation="silu", output_final_state=True,
                                         cu_seqlens=cu, **at)
        at = dict(initial_state=state, output_state=state, state_indices=idx)
        if cu is not None:
            at["cu_seqlens"] = cu
        if self.kind == "delta":
            q, k, v = [t.contiguous() for t in y.view(-1, 3, self.H, self.D).unbind(1)]
            call = gdn.gated_delta_rule_decode if cu is None else gdn.chunk_gated_delta_rule
            o, _ = call(q, k, v, self.g[tokens], self.beta[tokens], output_final_state=True,
                        use_qk_l2norm_in_kernel=True, **at)
            o = o.reshape(o.shape[0], -1)
        else:
            call = gdn.selective_scan_decode if cu is None else gdn.selective_scan
            o, _ = call(y, y, self.A, self.B[tokens], self.Cm[tokens], delta_softplus=True,
                        output_final_state=True, **at)
        return o @ self.head


@pytest.mark.parametrize("kind", ["delta", "scan"])
def test_beam_search_over_pools(kind):
    """Three steps of beam search: every beam's rows and scores are those of its own
    history run as a prompt."""
    m, B, K = Model(kind), 3, 4
    gen = torch.Generator().manual_seed(6)
    lens = [5, 1, 70]
    prompt = [torch.randint(m.V, (n,), generator=gen) for n in lens]
    pools = m.pools(B * K + 2)
    idx = torch.randperm(B * K + 2, generator=gen)[:B * K].to(torch.int32).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    lead = idx.view(B, K)[:, 0].contiguous()
    logits = m.run(torch.cat(prompt).cuda(), pools, lead, cu)[(cu[1:] - 1).long()]
    score, _, token = gdn.beam_select(logits[:, None], torch.zeros((B, 1), device="cuda"), K)
    for p in pools:  # one prompt, K beams
        gdn.state_pool_copy(p, lead.repeat_interleave(K - 1).contiguous(),
                            idx.view(B, K)[:, 1:].reshape(-1).contiguous())
    history = [[prompt[b].tolist() + [t] for t in token[b].tolist()] for b in range(B)]
    for _ in range(3):
        logits = m.run(token.reshape(-1).long(), pools, idx).view(B, K, -1)
        score, parent, token = gdn.beam_select(logits, score)
        idx = gdn.state_pool_reorder(pools, idx, parent)
        history = [[history[b][p] + [t] for p, t in zip(parent[b].tolist(), token[b].tolist())]
                   for b in range(B)]
    flat = [h for g in history for h in g]
    assert len(set(map(tuple, flat))) == B * K
    again = m.pools(B * K)
    cu = torch.tensor([0] + [len(h) - 1 for h in flat]).cumsum(0).to(torch.int32).cuda()
    every = m.run(torch.tensor(sum((h[:-1] for h in flat), [])).cuda(), again,
                  torch.arange(B * K, dtype=torch.int32, device="cuda"), cu)
    for p, q in zip(pools, again):
        # the same recurrence in fp32, a step at a time and in chunks
        assert torch.allclose(p[idx.long()], q, rtol=1e-3, atol=1e-3)
    logp = torch.log_softmax(every.double(), -1)
    for i, h in enumerate(flat):
        at, n = int(cu[i]), lens[i // K]
        want = sum(logp[at + j - 1, h[j]].item() for j in range(n, len(h)))
        assert abs(want - score.view(-1)[i].item()) <= 1e-2


def test_training_step_through_a_layer():
    """Gradients flow through the convolution and the scan behind it, as through
    their definitions in fp64."""
    lens, C, N = [30, 1, 0, 40], 12, 4
    c = L.conv_make(1, lens, C, 4)
    d = L.scan_make(2, lens, C, N)
    x, w, A = (t.clone().requires_grad_() for t in (c["x"], c["w"], d["A"]))
    y = gdn.short_convolution(x, w, c["bias"], "silu", cu_seqlens=c["cu"])
    out = gdn.selective_scan(y, d["delta"], A, d["B"], d["C"], z=d["z"], delta_softplus=True,
                             cu_seqlens=c["cu"])
    out.backward(d["dy"])
    n = {k: f64(v) for k, v in d.items() if k != "cu"}
    for k in ("D", "dbias", "h0", "dfinal"):
        n[k] = None
    outs, _, _, _ = L.conv_forward(f64(x), f64(w), f64(c["bias"]), lens, None, "silu")
    n["x"] = np.concatenate([o.v for o in outs])
    back = L.Scan(n, lens, True).backward()
    first = L.conv_backward(back["dx"].v, f64(x), f64(w), f64(c["bias"]), lens, None, None, "silu")
    # y and its gradient were rounded to fp32 on the way: a few 2^-24 of terms of
    # the order of the largest gradient each
    for got, want in ((A.grad, back["dA"]), (x.grad, first["dx"]), (w.grad, first["dw"])):
        scale = np.abs(want.v).max()
        assert np.abs(f64(got) - want.v).max() <= want.e.max() + 200 * 2.0 ** -24 * scale


def _calls():
    """Every operator once: (name, call that returns tensors)."""
    lens = [100, 3, 0, 200]
    c = L.conv_make(1, lens, 256, 4, BF16, BF16)
    d = L.scan_make(2, lens, 64, 16, 1, BF16)
    many = L.conv_make(3, [3] * 80, 64, 4)
    args = (d["x"], d["delta"], d["A"], d["B"], d["C"])
    logits = torch.randn((4, 4, 9000), device="cuda")
    scores = torch.randn((4, 4), device="cuda")
    pool = torch.randn((20, 64), device="cuda")
    idx = torch.arange(16, dtype=torch.int32, device="cuda")
    par = torch.randint(4, (4, 4), device="cuda").int()
    tup = lambda r: tuple(t for t in (r if isinstance(r, tuple) else (r,)) if t is not None)  # noqa: E731
    return {
        "conv": lambda: tup(gdn.short_convolution(c["x"], c["w"], c["bias"], "silu", c["h0"], True, c["cu"])),
        "conv many": lambda: tup(gdn.short_convolution(many["x"], many["w"], cu_seqlens=many["cu"])),
        "conv backward": lambda: tup(gdn.short_convolution_backward(
            c["dy"], c["x"], c["w"], c["bias"], "silu", cu_seqlens=c["cu"])),
        "conv decode": lambda: tup(gdn.short_convolution_decode(c["x"], c["w"])),
        "scan": lambda: tup(gdn.selective_scan(*args, z=d["z"], delta_softplus=True, initial_state=d["h0"],
                                               output_final_state=True, cu_seqlens=d["cu"])),
        "scan backward": lambda: tup(gdn.selective_scan_backward(
            d["dy"], *args, D=d["D"], z=d["z"], delta_softplus=True, initial_state=d["h0"],
            cu_seqlens=d["cu"], output_dinitial_state=True)),
        "scan decode": lambda: tup(gdn.selective_scan_decode(*args, delta_softplus=True)),
        "select": lambda: gdn.beam_select(logits, scores),
        "reorder": lambda: (lambda p: (p, gdn.state_pool_reorder(p, idx, par)))(pool.clone()),
    }


NAMES = ["conv", "conv many", "conv backward", "conv decode", "scan", "scan backward", "scan decode",
         "select", "reorder"]


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name):
    """Captured, replayed several times with eager calls of the same operator
    between the replays."""
    call = _calls()[name]
    want = call()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = call()
    for _ in range(4):
        for t in held:
            t.zero_()
        graph.replay()
        other = call()
        torch.cuda.synchronize()
        for a, b, c in zip(held, want, other):
            assert L.same(a, b) and L.same(c, b)


@pytest.mark.parametrize("name", NAMES)
def test_threads_and_streams(name):
    """Two threads on streams of their own, and two on one stream: workspaces are
    the streams' own, calls' kernels stay together."""
    call = _calls()[name]
    want = call()
    torch.cuda.synchronize()
    shared, bad = torch.cuda.Stream(), []

    def work(stream):
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = call()
                stream.synchronize()
                if not all(L.same(a, b) for a, b in zip(got, want)):
                    bad.append(name)

    threads = [threading.Thread(target=work, args=(s,))
               for s in (torch.cuda.Stream(), torch.cuda.Stream(), shared, shared)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_workspaces():
    """A workspace of the caller's, too small or not; NaN in it changes nothing."""
    d = L.scan_make(3, [300], 64, 16)
    args = (d["x"], d["delta"], d["A"], d["B"], d["C"])
    more = {"delta_softplus": True}
    want = gdn.selective_scan(*args, **more)
    back = gdn.selective_scan_backward(d["dy"], *args, **more)
    assert torch.isfinite(want).all()
    for size in (1, 1 << 24):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        assert L.same(gdn.selective_scan(*args, workspace=ws, **more), want)
        ws.fill_(255)
        for a, b in zip(gdn.selective_scan_backward(d["dy"], *args, workspace=ws, **more), back):
            assert a is b is None or L.same(a, b)
    c = L.conv_make(4, [5] * 70, 64, 4)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    out = gdn.short_convolution(c["x"], c["w"], cu_seqlens=c["cu"], workspace=ws)
    assert torch.equal(out, gdn.short_convolution(c["x"], c["w"], cu_seqlens=c["cu"]))
    with pytest.raises(ValueError):
        gdn.selective_scan(*args, workspace=ws.float())


def test_written_versions_and_captured_gradients():
    c = L.conv_make(5, [6, 4], 16, 4)
    d = L.scan_make(6, [6, 4], 16, 4)
    pool, states = torch.zeros((4, 3, 16), device="cuda"), torch.zeros((4, 16, 4), device="cuda")
    idx = torch.tensor([1, 2], device="cuda")
    args = (d["x"], d["delta"], d["A"], d["B"], d["C"])
    for t, call in (
            (pool, lambda: gdn.short_convolution(c["x"], c["w"], initial_state=pool, output_final_state=True,
                                                 cu_seqlens=c["cu"], output_state=pool, state_indices=idx)),
            (pool, lambda: gdn.short_convolution_decode(c["x"][:2], c["w"], initial_state=pool,
                                                        output_state=pool, state_indices=idx)),
            (states, lambda: gdn.selective_scan(*args, initial_state=states, output_final_state=True,
                                                cu_seqlens=d["cu"], output_state=states, state_indices=idx)),
            (pool, lambda: gdn.state_pool_reorder([states, pool], idx, torch.zeros((1, 2), dtype=torch.int64,
                                                                                   device="cuda")))):
        version = t._version
        call()
        assert t._version > version
    x = c["x"].clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        held = c["x"] * 1.0
        for call in (lambda: gdn.short_convolution(x, c["w"]),
                     lambda: gdn.selective_scan(x, *args[1:])):
            with pytest.raises(RuntimeError):
                call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, c["x"])
