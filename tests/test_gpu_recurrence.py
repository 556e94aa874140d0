"""GPU tests of the gated linear recurrence (forward, backward, decode) against
its definition in fp64, with elementwise bounds derived from the roundings a
value passes (tests/recurrence_testlib.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    gated_linear_recurrence, gated_linear_recurrence_backward, gated_linear_recurrence_decode)
from tests import recurrence_testlib as R  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


LENS = {
    "one": [1],
    "tile": [64],
    "tile+1": [65],
    "ragged": [130, 20, 0, 300, 0, 64, 1],
    "edges": [63, 1, 64, 128, 0, 0, 5, 59],
    "long": [5000],
    "ones": [1] * 70,
    "many": [3, 0, 17, 1, 90, 0, 0, 2] * 12,
}


def _both(d, lens, **kw):
    """Forward with kept states, then backward; checks everything."""
    T, H, D = d["x"].shape
    out, fin, kept = gated_linear_recurrence(
        d["x"], d["g"], initial_state=d["h0"], output_final_state=True, cu_seqlens=d["cu"],
        return_chunk_states=True)
    dx, dg, dh0 = gated_linear_recurrence_backward(
        d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)
    x, g, h0 = R.f64(d["x"]), R.f64(d["g"]), R.f64(d["h0"])
    h, err, final, ferr = R.forward(x, g, lens, h0)
    n = sum(lens)
    R.check("out", out[:n], h[:n], err[:n], out.dtype)
    R.check("final", fin, final, ferr, F32)
    w = R.backward(R.f64(d["dy"]), x, g, lens, h0, R.f64(d["dfinal"]))
    R.check("dx", dx, *w["dx"], dx.dtype)
    R.check("dg", dg, *w["dg"], dg.dtype)
    R.check("dh0", dh0, *w["dh0"], F32)
    return out, fin, kept, dx, dg, dh0


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype,gate,per_head", [
    (F32, F32, False), (BF16, F32, False), (F16, F16, False), (BF16, BF16, True),
    (F32, F32, True), (F16, F32, True)])
def test_forward_and_backward(lens, dtype, gate, per_head):
    d = R.make(1, LENS[lens], 3, 32, dtype, gate, per_head)
    _both(d, LENS[lens])


@pytest.mark.parametrize("H,D", [(1, 1), (1, 3), (5, 7), (3, 85), (1, 257), (2, 128), (9, 64)])
@pytest.mark.parametrize("dtype,gate", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)])
def test_odd_widths(H, D, dtype, gate):
    d = R.make(2, [70, 0, 1, 66], H, D, dtype, gate)
    _both(d, [70, 0, 1, 66])


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H", [1, 5, 16])
def test_head_gate_sizes(H, D):
    d = R.make(3, [100, 31], H, D, BF16, F32, True)
    _both(d, [100, 31])


def test_slow_gates_over_a_long_chain():
    # gates close to one over 300 tiles: the carry matters at every token and
    # comes from far behind the look-back window
    lens = [19200]
    d = R.make(4, lens, 1, 64)
    d["g"] = (1 - 1e-4 * torch.rand_like(d["g"])).contiguous()
    _both(d, lens)


def test_zero_gates_and_unit_gates():
    lens = [200, 100]
    d = R.make(5, lens, 2, 32)
    d["g"][::3] = 0.0
    d["g"][1::3] = 1.0
    _both(d, lens)


def test_no_initial_state_no_final_state_one_sequence():
    d = R.make(6, [333], 4, 32, BF16, h0=False)
    out = gated_linear_recurrence(d["x"], d["g"])
    h, err, _, _ = R.forward(R.f64(d["x"]), R.f64(d["g"]), [333])
    R.check("out", out, h, err, BF16)
    dx, dg = gated_linear_recurrence_backward(d["dy"], d["x"], d["g"])
    w = R.backward(R.f64(d["dy"]), R.f64(d["x"]), R.f64(d["g"]), [333])
    R.check("dx", dx, *w["dx"], BF16)
    R.check("dg", dg, *w["dg"], F32)


@pytest.mark.parametrize("n", [5, 100])
def test_rows_outside_the_sequences(n):
    """Rows before the first and behind the last sequence: outputs untouched,
    gradients zero, whatever the rows hold."""
    lens = [7] * n
    begin, tail = 70, 131
    d = R.make(7, [begin] + lens, 2, 32, tail=tail)
    cu = torch.tensor([begin] + [7] * n).cumsum(0).to(torch.int32).cuda()
    x, g, dy = d["x"], d["g"], d["dy"]
    stop = begin + 7 * n
    for t in (x, g, dy):
        t[:begin] = float("nan")
        t[stop:] = float("inf")
    h0, dfin = d["h0"][1:].contiguous(), d["dfinal"][1:].contiguous()
    out = torch.full_like(x, 7.5)
    res, fin, kept = gated_linear_recurrence(x, g, initial_state=h0, output_final_state=True,
                                             cu_seqlens=cu, output=out, return_chunk_states=True)
    assert res is out
    assert torch.all(out[:begin] == 7.5) and torch.all(out[stop:] == 7.5)
    h, err, final, ferr = R.forward(R.f64(x), R.f64(g), lens, R.f64(h0), begin)
    R.check("out", out[begin:stop], h[begin:stop], err[begin:stop], F32)
    R.check("final", fin, final, ferr, F32)
    dx, dg, dh0 = gated_linear_recurrence_backward(
        dy, x, g, initial_state=h0, dfinal_state=dfin, cu_seqlens=cu, chunk_states=kept,
        output_dinitial_state=True)
    w = R.backward(np.nan_to_num(R.f64(dy), posinf=0), np.nan_to_num(R.f64(x), posinf=0),
                   np.nan_to_num(R.f64(g), posinf=0), lens, R.f64(h0), R.f64(dfin), begin)
    for name, got in (("dx", dx), ("dg", dg), ("dh0", dh0)):
        R.check(name, got, *w[name], F32)
    assert torch.all(dx[:begin] == 0) and torch.all(dx[stop:] == 0)
    assert torch.all(dg[:begin] == 0) and torch.all(dg[stop:] == 0)


def test_nan_and_infinity_stay_in_their_sequence():
    lens = [40, 100, 0, 30, 200]
    d = R.make(8, lens, 2, 32)
    d["x"][10] = float("nan")
    d["x"][60] = float("inf")
    d["h0"][3] = float("nan")
    d["g"][175] = float("inf")
    d["dy"][12] = float("nan")
    d["dy"][100] = float("inf")
    out, fin, kept = gated_linear_recurrence(
        d["x"], d["g"], initial_state=d["h0"], output_final_state=True, cu_seqlens=d["cu"],
        return_chunk_states=True)
    dx, dg, dh0 = gated_linear_recurrence_backward(
        d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)
    assert torch.isfinite(out[:10]).all() and torch.isnan(out[10:40]).all()
    assert torch.isfinite(out[40:60]).all() and torch.isinf(out[60:140]).all()
    assert torch.isnan(out[140:170]).all()
    assert torch.isfinite(out[170:175]).all() and not torch.isfinite(out[175:]).any()
    # the empty sequence's final state is its start
    assert torch.equal(fin[2], d["h0"][2])
    assert torch.isfinite(dx[13:40]).all() and torch.isnan(dx[:13]).all()
    assert torch.isfinite(dx[101:140]).all() and not torch.isfinite(dx[40:101]).any()
    assert torch.isfinite(dx[140:170]).all()
    assert torch.isfinite(dx[175:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16, E4M3, E5M2])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_pool_states(dtype, index):
    lens = [100, 0, 1, 64, 200]
    d = R.make(9, lens, 3, 32, BF16)
    idx = torch.tensor([7, 2, 9, 0, 4], dtype=index, device="cuda")
    pool = torch.randn((11, 3, 32), device="cuda").to(dtype)
    before = pool.clone()
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out, fin = gated_linear_recurrence(
        d["x"], d["g"], initial_state=pool, output_final_state=True, cu_seqlens=d["cu"],
        output_state=pool, state_indices=idx, status=st)
    assert fin is pool and st.item() == 0
    rows = idx.tolist()
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), lens,
                                    R.f64(before)[rows])
    R.check("out", out, h, err, BF16)
    R.check("final", pool[idx.long()].float(), final, ferr, dtype)
    assert torch.equal(pool[2].float(), before[2].float())  # the empty sequence's row
    others = [r for r in range(11) if r not in rows]
    assert torch.equal(pool[others].view(torch.uint8) if dtype in (E4M3, E5M2) else pool[others],
                       before[others].view(torch.uint8) if dtype in (E4M3, E5M2)
                       else before[others])


@pytest.mark.parametrize("n", [4, 80])
def test_bad_state_indices(n):
    """An index out of range: status bit, a start from zero, nothing written."""
    lens = [9] * n
    d = R.make(10, lens, 2, 32)
    idx = torch.arange(n, dtype=torch.int64, device="cuda")
    idx[1], idx[2] = n + 5, -1
    pool = torch.randn((n, 2, 32), device="cuda")
    before = pool.clone()
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out, _ = gated_linear_recurrence(d["x"], d["g"], initial_state=pool, output_final_state=True,
                                     cu_seqlens=d["cu"], output_state=pool, state_indices=idx,
                                     status=st)
    assert st.item() == 4
    h0 = R.f64(before).copy()
    h0[1] = h0[2] = 0
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), lens, h0)
    R.check("out", out, h, err, F32)
    R.check("final", pool[3:], final[3:], ferr[3:], F32)
    assert torch.equal(pool[1:3], before[1:3])


@pytest.mark.parametrize("n", [3, 90])
def test_bad_cu_seqlens_set_the_status(n):
    """Offsets that fall or leave [0, T] count as their running maximum,
    clamped; nothing is read or written out of range."""
    T = 10 * n
    cu = torch.arange(0, T + 1, 10, dtype=torch.int64)
    cu[1], cu[2] = 25, 20
    cu[-1] = T + 1000
    d = R.make(11, [T], 2, 32)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    h0 = torch.randn((n, 2, 32), device="cuda")
    out, fin = gated_linear_recurrence(d["x"], d["g"], initial_state=h0, output_final_state=True,
                                       cu_seqlens=cu.cuda(), status=st)
    assert st.item() == 1
    real = np.maximum.accumulate(np.clip(cu.numpy(), 0, T))
    lens = np.diff(real).tolist()
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), lens, R.f64(h0))
    R.check("out", out, h, err, F32)
    R.check("final", fin, final, ferr, F32)


def test_no_tokens():
    x = torch.empty((0, 2, 32), device="cuda")
    g = torch.empty((0, 2, 32), device="cuda")
    h0 = torch.randn((3, 2, 32), device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out, fin = gated_linear_recurrence(x, g, initial_state=h0, output_final_state=True,
                                       cu_seqlens=cu, status=st)
    assert out.shape == x.shape and torch.equal(fin, h0) and st.item() == 0
    dfin = torch.randn_like(h0)
    dx, dg, dh0 = gated_linear_recurrence_backward(x, x, g, initial_state=h0, dfinal_state=dfin,
                                                   cu_seqlens=cu, output_dinitial_state=True)
    assert dx.shape == x.shape and dg.shape == g.shape and torch.equal(dh0, dfin)
    # no sequences at all
    out, fin = gated_linear_recurrence(x, g, output_final_state=True, cu_seqlens=cu[:1])
    assert fin.shape == (0, 2, 32)
    out, fin = gated_linear_recurrence_decode(x, g)
    assert out.shape == x.shape and fin.shape == (0, 2, 32)


@pytest.mark.parametrize("dtype,gate", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("off,pad", [(0, 64), (3, 1), (1, 0)])
def test_strided_tokens(dtype, gate, off, pad):
    """x, g and doutput as slices of wider rows, at any offset."""
    lens = [90, 45]
    d = R.make(12, lens, 3, 32, dtype, gate)
    T, C = 135, 96

    def slot(t):
        wide = torch.full((T, off + C + pad), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, off:off + C] = t.reshape(T, C)
        return wide[:, off:off + C].view(T, 3, 32) if pad == 0 and off == 0 \
            else wide[:, off:off + C].unflatten(1, (3, 32))

    ref = _both(d, lens)
    got = _both(dict(d, x=slot(d["x"]), g=slot(d["g"]), dy=slot(d["dy"])), lens)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("off", [0, 1, 4])
def test_strided_head_gates(off):
    """Head gates as columns of a wider projection, x off a vector boundary."""
    lens = [90, 45]
    d = R.make(12, lens, 3, 64, F16, F32, True)
    ref = _both(d, lens)
    gw = torch.full((135, 11), float("nan"), device="cuda")
    gw[:, off:off + 3] = d["g"]
    xw = torch.full((135, 200), float("nan"), dtype=F16, device="cuda")
    xw[:, off:off + 192] = d["x"].reshape(135, 192)
    got = _both(dict(d, g=gw[:, off:off + 3], x=xw[:, off:off + 192].unflatten(1, (3, 64))), lens)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_thousands_of_sequences():
    """More sequences than a workgroup has threads, most of them empty, several
    ending in one tile, long runs of empty ones."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 3, 3000)
    lens[rng.random(3000) < 0.6] = 0
    lens[1000:2200] = 0
    lens[2300] = 150
    lens = lens.tolist()
    d = R.make(13, lens, 1, 40)
    _both(d, lens)


@pytest.mark.parametrize("n", [63, 64, 65, 6000])
def test_all_but_one_sequence_empty(n):
    """Empty sequences' states are copied by workgroups of their own: 64 to a
    workgroup, and more sequences than those workgroups hold at once."""
    lens = [0] * n
    lens[n // 3] = 5
    d = R.make(19, lens, 2, 150)
    _both(d, lens)
    # from a pool of another type, an index out of range among them
    idx = torch.randperm(n + 2)[:n].to(torch.int32)
    idx[n - 1] = n + 2
    pool = torch.randn((n + 2, 2, 150), device="cuda").to(BF16)
    final = torch.full((n + 2, 2, 150), 7.0, device="cuda")
    gated_linear_recurrence(d["x"], d["g"], initial_state=pool, output_final_state=True,
                            cu_seqlens=d["cu"], output_state=final, state_indices=idx.cuda())
    want = torch.full_like(final, 7.0)
    for i in range(n - 1):
        if lens[i] == 0:
            want[idx[i]] = pool[idx[i]].float()
    row = int(idx[n // 3])
    want[row] = final[row]
    assert torch.equal(final, want)


def test_output_in_place_of_x():
    lens = [100, 300]
    d = R.make(14, lens, 3, 32, BF16)
    want = gated_linear_recurrence(d["x"], d["g"], initial_state=d["h0"], cu_seqlens=d["cu"])
    x = d["x"].clone()
    got = gated_linear_recurrence(x, d["g"], initial_state=d["h0"], cu_seqlens=d["cu"], output=x)
    assert got is x and torch.equal(got, want)


def test_sequences_that_share_a_start_row():
    """Without a final state several sequences may start from one pool row."""
    lens = [10, 70, 5]
    d = R.make(15, lens, 2, 32)
    pool = torch.randn((4, 2, 32), device="cuda")
    idx = torch.tensor([2, 2, 0], dtype=torch.int32, device="cuda")
    out = gated_linear_recurrence(d["x"], d["g"], initial_state=pool, cu_seqlens=d["cu"],
                                  state_indices=idx)
    h, err, _, _ = R.forward(R.f64(d["x"]), R.f64(d["g"]), lens, R.f64(pool)[[2, 2, 0]])
    R.check("out", out, h, err, F32)


def test_workspace_of_the_caller():
    """A workspace that holds anything, reused by calls of other shapes."""
    ws = torch.randint(0, 256, (1 << 22,), dtype=torch.uint8, device="cuda")
    for lens, seed in (([700, 20], 16), ([5] * 100, 17), ([130], 18)):
        d = R.make(seed, lens, 3, 32)
        ref = _run_all(d)
        out, fin, kept = gated_linear_recurrence(
            d["x"], d["g"], initial_state=d["h0"], output_final_state=True, cu_seqlens=d["cu"],
            return_chunk_states=True, workspace=ws)
        got = (out, fin) + gated_linear_recurrence_backward(
            d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
            cu_seqlens=d["cu"], output_dinitial_state=True, workspace=ws)
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_strided_pool_rows():
    """One layer's slice of a [rows, layers, H, D] pool."""
    lens = [30, 70]
    d = R.make(13, lens, 3, 32)
    big = torch.randn((6, 4, 3, 32), device="cuda")
    before = big.clone()
    idx = torch.tensor([5, 1], dtype=torch.int32, device="cuda")
    gated_linear_recurrence(d["x"], d["g"], initial_state=big[:, 2], output_final_state=True,
                            cu_seqlens=d["cu"], output_state=big[:, 2], state_indices=idx)
    _, _, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), lens, R.f64(before[[5, 1], 2]))
    R.check("final", big[[5, 1], 2], final, ferr, F32)
    big[[5, 1], 2] = before[[5, 1], 2]
    assert torch.equal(big, before)


def test_backward_forms_the_states_itself():
    """Without the kept states the same numbers come out."""
    for lens in ([50], [700, 3, 0, 129]):
        d = R.make(14, lens, 3, 85, BF16)
        ref = _both(d, lens)
        got = gated_linear_recurrence_backward(
            d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
            cu_seqlens=d["cu"], output_dinitial_state=True)
        for a, b in zip(ref[3:], got):
            assert torch.equal(a, b)


def test_repeatable_bit_for_bit():
    lens = [4000, 1, 3000]
    d = R.make(15, lens, 16, 128, BF16)
    ref = _run_all(d)
    for _ in range(5):
        for a, b in zip(ref, _run_all(d)):
            assert torch.equal(a, b)


def _run_all(d):
    out, fin, kept = gated_linear_recurrence(
        d["x"], d["g"], initial_state=d["h0"], output_final_state=True, cu_seqlens=d["cu"],
        return_chunk_states=True)
    return (out, fin) + gated_linear_recurrence_backward(
        d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)


def test_two_streams_at_once():
    """Two long chains side by side: each stream has a workspace of its own."""
    d1 = R.make(16, [6000], 8, 128, BF16)
    d2 = R.make(17, [3000, 5000], 8, 128, BF16)
    ref1, ref2 = _run_all(d1), _run_all(d2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got1, got2 = [], []
    for _ in range(3):
        with torch.cuda.stream(s1):
            got1.append(_run_all(d1))
        with torch.cuda.stream(s2):
            got2.append(_run_all(d2))
    torch.cuda.synchronize()
    for ref, got in ((ref1, got1), (ref2, got2)):
        for g in got:
            for a, b in zip(ref, g):
                assert torch.equal(a, b)


def test_threads_on_one_stream():
    """Threads that share a stream share its workspace; a call's kernels stay
    together."""
    import threading
    ds = [R.make(60 + i, [900 + 64 * i, 300], 2, 64, BF16) for i in range(4)]
    refs = [_run_all(d) for d in ds]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(50):
            if not all(torch.equal(a, b) for a, b in zip(refs[i], _run_all(ds[i]))):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_graph_replay():
    """A training step captured once and replayed on new inputs, with eager
    work between the replays."""
    lens = [700, 0, 300]
    d = R.make(18, lens, 4, 64, BF16)
    _run_all(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run_all(d)
    torch.cuda.current_stream().wait_stream(side)
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = _run_all(d)
    with torch.cuda.graph(second):
        res2 = _run_all(d)
    for seed in range(20, 24):
        n = R.make(seed, lens, 4, 64, BF16)
        for k in ("x", "g", "h0", "dy", "dfinal"):
            d[k].copy_(n[k])
        graph.replay()
        second.replay()
        eager = _run_all(n)
        torch.cuda.synchronize()
        for a, b, c in zip(eager, res, res2):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_gradients_against_differences():
    """d loss / d input by central differences of the fp64 definition, for the
    loss sum(w out) + sum(v final)."""
    lens = [5, 0, 3]
    d = R.make(19, lens, 2, 32, per_head=True)
    _, _, dx, dg, dh0 = _run_all(d)
    x, g, h0 = R.f64(d["x"]), R.f64(d["g"]), R.f64(d["h0"])
    w, v = R.f64(d["dy"]), R.f64(d["dfinal"])

    def loss():
        h, _, final, _ = R.forward(x, g, lens, h0)
        return (w * h).sum() + (v * final).sum()

    rng = np.random.default_rng(0)
    step = 1e-5
    for name, arr, grad in (("x", x, dx), ("g", g, dg), ("h0", h0, dh0)):
        got = R.f64(grad)
        for flat in rng.choice(arr.size, 12, replace=False):
            at = np.unravel_index(flat, arr.shape)
            keep = arr[at]
            arr[at] = keep + step
            up = loss()
            arr[at] = keep - step
            down = loss()
            arr[at] = keep
            # the loss is at most quadratic in the step for x and h0, cubic
            # terms of g are below step^2 times a few hundred
            num = (up - down) / (2 * step)
            assert abs(num - got[at]) <= 1e-5 * (1 + abs(num)), (name, at, num, got[at])


# ------------------------------------------------------------------ autograd

@pytest.mark.parametrize("gate,per_head", [(F32, False), (BF16, True)])
def test_autograd_matches_the_explicit_call(gate, per_head):
    lens = [100, 0, 31]
    d = R.make(30, lens, 3, 32, BF16, gate, per_head)
    ref = _run_all(d)
    leaves = [d[k].clone().requires_grad_() for k in ("x", "g", "h0")]
    out, fin = gated_linear_recurrence(leaves[0], leaves[1], initial_state=leaves[2],
                                       output_final_state=True, cu_seqlens=d["cu"])
    assert torch.equal(out, ref[0]) and torch.equal(fin, ref[1])
    torch.autograd.backward([out, fin], [d["dy"], d["dfinal"]])
    for leaf, want in zip(leaves, ref[2:]):
        assert torch.equal(leaf.grad, want)


def test_autograd_partial_and_broadcast_gradients():
    """Only out used, an expanded incoming gradient, an initial state shared
    by the sequences (its gradient sums over them), no gradient for g."""
    lens = [20, 30]
    d = R.make(31, lens, 2, 32)
    x = d["x"].clone().requires_grad_()
    one = torch.randn((1, 2, 32), device="cuda", requires_grad=True)
    out = gated_linear_recurrence(x, d["g"], initial_state=one.expand(2, 2, 32),
                                  cu_seqlens=d["cu"])
    out.sum().backward()
    ones = np.ones(x.shape)
    w = R.backward(ones, R.f64(x), R.f64(d["g"]), lens, R.f64(one.expand(2, 2, 32)))
    R.check("dx", x.grad, *w["dx"], F32)
    v, e = w["dh0"]
    R.check("dh0", one.grad, v.sum(0, keepdims=True), e.sum(0, keepdims=True)
            + R.U32 * np.abs(v).sum(0, keepdims=True), F32)
    # only the final state used
    x2 = d["x"].clone().requires_grad_()
    _, fin = gated_linear_recurrence(x2, d["g"], output_final_state=True, cu_seqlens=d["cu"])
    fin.sum().backward()
    w = R.backward(0 * ones, R.f64(x2), R.f64(d["g"]), lens, None, np.ones((2, 2, 32)))
    R.check("dx", x2.grad, *w["dx"], F32)


def test_autograd_refusals(monkeypatch):
    d = R.make(32, [10], 2, 32)
    x = d["x"].clone().requires_grad_()
    for kw in (dict(output=torch.empty_like(d["x"])), dict(return_chunk_states=True),
               dict(status=torch.zeros(1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            gated_linear_recurrence(x, d["g"], **kw)
    with torch.no_grad():
        gated_linear_recurrence(x, d["g"], output=torch.empty_like(d["x"]))
    out = gated_linear_recurrence(x, d["g"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError):
        gated_linear_recurrence(x, d["g"])
    with pytest.raises(RuntimeError):
        out.sum().backward()


# -------------------------------------------------------------------- decode

@pytest.mark.parametrize("dtype,gate,per_head", [
    (F32, F32, False), (BF16, F32, False), (BF16, BF16, True), (F16, F16, False)])
@pytest.mark.parametrize("N,H,D", [(1, 1, 32), (37, 3, 64), (300, 2, 128)])
def test_decode(dtype, gate, per_head, N, H, D):
    d = R.make(40, [1] * N, H, D, dtype, gate, per_head)
    out, fin = gated_linear_recurrence_decode(d["x"], d["g"], initial_state=d["h0"])
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), [1] * N, R.f64(d["h0"]))
    R.check("out", out, h, err, dtype)
    R.check("final", fin, final, ferr, F32)


@pytest.mark.parametrize("dtype", [F32, BF16, F16, E4M3, E5M2])
def test_decode_pool_in_place(dtype):
    N = 20
    d = R.make(41, [1] * N, 5, 7, F16)
    idx = torch.randperm(33)[:N].to(torch.int32).cuda()
    pool = torch.randn((33, 5, 7), device="cuda").to(dtype)
    before = pool.clone()
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out, fin = gated_linear_recurrence_decode(d["x"], d["g"], initial_state=pool,
                                              output_state=pool, state_indices=idx, status=st)
    assert fin is pool and st.item() == 0
    rows = idx.tolist()
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), [1] * N, R.f64(before)[rows])
    R.check("out", out, h, err, F16)
    R.check("final", pool.float()[rows], final, ferr, dtype)
    others = [r for r in range(33) if r not in rows]
    assert torch.equal(pool.float()[others], before.float()[others])


def test_decode_bad_index_and_strides():
    N = 6
    d = R.make(42, [1] * N, 2, 32)
    wide = torch.full((N, 70), float("nan"), device="cuda")
    wide[:, 3:67] = d["x"].reshape(N, 64)
    x = wide[:, 3:67].unflatten(1, (2, 32))
    idx = torch.tensor([0, 9, 2, -1, 1, 3], dtype=torch.int64, device="cuda")
    pool = torch.randn((4, 2, 32), device="cuda")
    before = pool.clone()
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out, _ = gated_linear_recurrence_decode(x, d["g"], initial_state=pool, output_state=pool,
                                            state_indices=idx, status=st)
    assert st.item() == 4
    h0 = np.zeros((N, 2, 32))
    good = [0, 2, 4, 5]
    h0[good] = R.f64(before)[[0, 2, 1, 3]]
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), [1] * N, h0)
    R.check("out", out, h, err, F32)
    R.check("final", pool[[0, 2, 1, 3]], final[good], ferr[good], F32)


def test_decode_continues_a_prefill():
    """Prefill n tokens and decode m more: the recurrence over all of them."""
    n, m, N = 70, 5, 3
    d = R.make(43, [n + m] * N, 2, 32)
    x, g = (d[k].view(N, n + m, 2, 32) for k in ("x", "g"))
    pool = torch.zeros((8, 2, 32), device="cuda")
    idx = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
    pool[idx.long()] = d["h0"]
    cu = torch.arange(0, N * n + 1, n, dtype=torch.int32, device="cuda")
    gated_linear_recurrence(x[:, :n].reshape(N * n, 2, 32), g[:, :n].reshape(N * n, 2, 32),
                            initial_state=pool, output_final_state=True, cu_seqlens=cu,
                            output_state=pool, state_indices=idx)
    h, err, final, ferr = R.forward(R.f64(d["x"]), R.f64(d["g"]), [n + m] * N, R.f64(d["h0"]))
    h, err = h.reshape(N, n + m, 2, 32), err.reshape(N, n + m, 2, 32)
    for j in range(m):
        out, _ = gated_linear_recurrence_decode(x[:, n + j].contiguous(), g[:, n + j].contiguous(),
                                                initial_state=pool, output_state=pool,
                                                state_indices=idx)
        R.check("out", out, h[:, n + j], err[:, n + j], F32)
    R.check("final", pool[idx.long()], final, ferr, F32)


# ------------------------------------------------------------------ refusals

def test_refused_on_the_device():
    d = R.make(50, [10, 6], 2, 32, BF16)
    x, g, h0 = d["x"], d["g"], d["h0"]
    bad = [
        dict(x=x.to(E4M3)), dict(x=x[0]), dict(g=g.half()), dict(g=g[:, :1]),
        dict(x=x.transpose(1, 2).contiguous().transpose(1, 2)),
        dict(x=x[:1].expand(16, 2, 32)),
        dict(cu_seqlens=d["cu"].float()), dict(cu_seqlens=d["cu"].cpu()),
        dict(initial_state=h0[:1]), dict(initial_state=h0.double()),
        dict(output=torch.empty((16, 2, 32), device="cuda")),
        dict(output_final_state=True, output_state=torch.empty((3, 2, 32), device="cuda")),
        dict(output_final_state=True,
             output_state=torch.empty((1, 2, 32), device="cuda").expand(2, 2, 32)),
        dict(state_indices=torch.zeros(2, dtype=torch.int32, device="cuda")),
        dict(status=torch.zeros(1, device="cuda")),
        dict(workspace=torch.zeros(8, device="cuda")),
    ]
    for kw in bad:
        args = dict(x=x, g=g, cu_seqlens=d["cu"])
        args.update(kw)
        with pytest.raises(ValueError):
            gated_linear_recurrence(args.pop("x"), args.pop("g"), **args)
    with pytest.raises(ValueError):  # a head gate needs a head size of 32, 64 or 128
        gated_linear_recurrence(torch.zeros((4, 2, 48), device="cuda"),
                                torch.ones((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        gated_linear_recurrence_backward(d["dy"].float(), x, g, cu_seqlens=d["cu"])
    with pytest.raises(ValueError):
        gated_linear_recurrence_backward(d["dy"], x, g, cu_seqlens=d["cu"],
                                         chunk_states=torch.zeros((2, 2, 32), device="cuda"))
    with pytest.raises(ValueError):
        gated_linear_recurrence_decode(x, g, state_indices=torch.zeros(
            3, dtype=torch.int32, device="cuda"), initial_state=h0, output_state=h0)
