"""GPU tests of the selective scan against its definition in fp64: bounds of
sequences and tiles, states, pools, groups, types, gradients, decode steps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    _native as nat, selective_scan, selective_scan_backward, selective_scan_decode)
from tests import layers_testlib as L  # noqa: E402
from tests.recurrence_testlib import f64  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
GRADS = ("dx", "ddelta", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")
FP32_GRADS = ("dA", "dD", "dbias", "dh0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _args(d):
    return d["x"], d["delta"], d["A"], d["B"], d["C"]


def _layer(d, plus):
    return {"D": d["D"], "z": d["z"], "delta_bias": d["dbias"], "delta_softplus": plus}


def _want(d, lens, plus, begin=0):
    return L.Scan({k: f64(v) for k, v in d.items() if k != "cu"}, lens, plus, begin)


def _drop(d, *names):
    return dict(d, **{n: None for n in names})


# (lengths, channels, states, groups, type, softplus)
CASES = [
    ([1], 1, 1, 1, F32, True), ([0], 3, 4, 1, F32, True), ([0, 2, 1, 0, 15, 16, 17], 5, 3, 1, F32, True),
    ([130, 20, 300, 0, 64, 1], 8, 16, 1, F32, True), ([70, 9], 70, 16, 1, BF16, False),
    ([33, 40], 12, 8, 3, F16, True), ([50], 130, 5, 2, F32, False), ([40, 30], 6, 32, 1, BF16, True),
    ([37, 20], 4, 64, 2, F32, True), ([21], 3, 33, 1, F16, False), ([1] * 63, 4, 16, 1, F32, True),
    ([2, 0, 5] * 30, 3, 16, 1, BF16, True), ([3] * 64, 65, 2, 1, F32, True),
]


@pytest.mark.parametrize("lens,C,N,G,dtype,plus", CASES)
def test_forward(lens, C, N, G, dtype, plus):
    d = L.scan_make(C + N, lens, C, N, G, dtype, plus)
    out, final = selective_scan(*_args(d), **_layer(d, plus), initial_state=d["h0"],
                                output_final_state=True, cu_seqlens=d["cu"])
    want = _want(d, lens, plus)
    L.check("out", out, want.out, dtype)
    for i in range(len(lens)):
        L.check("final %d" % i, final[i], want.final[i], F32)
    few = _drop(d, "D", "z", "dbias", "h0")
    out = selective_scan(*_args(d), delta_softplus=plus, cu_seqlens=d["cu"])
    L.check("plain out", out, _want(few, lens, plus).out, dtype)


def _check_backward(d, lens, plus, dtype, got, begin=0, **more):
    want = _want(d, lens, plus, begin).backward()
    for name, g in zip(GRADS, got):
        if g is None:
            assert want.get(name) is None, name
            continue
        L.check(name, g, want[name], F32 if name in FP32_GRADS else dtype)


@pytest.mark.parametrize("lens,C,N,G,dtype,plus", CASES)
def test_backward(lens, C, N, G, dtype, plus):
    d = L.scan_make(2 * C + N, lens, C, N, G, dtype, plus)
    _, kept = selective_scan(*_args(d), **_layer(d, plus), initial_state=d["h0"], cu_seqlens=d["cu"],
                             return_chunk_states=True)
    grads = [selective_scan_backward(d["dy"], *_args(d), **_layer(d, plus), initial_state=d["h0"],
                                     dfinal_state=d["dfinal"], cu_seqlens=d["cu"], chunk_states=k,
                                     output_dinitial_state=True) for k in (kept, kept, None)]
    # the same from the same states, bit for bit; states formed again are composed
    # in another order
    _check_backward(d, lens, plus, dtype, grads[0])
    for a, b in zip(grads[0], grads[1]):
        assert L.same(a, b)
    _check_backward(d, lens, plus, dtype, grads[2])
    few = _drop(d, "D", "z", "dbias", "h0", "dfinal")
    got = selective_scan_backward(d["dy"], *_args(d), delta_softplus=plus, cu_seqlens=d["cu"])
    assert len(got) == 8 and got[5] is None and got[6] is None and got[7] is None
    _check_backward(few, lens, plus, dtype, got)


@pytest.mark.parametrize("lens,C,N,G,dtype", [([70, 9], 70, 16, 1, BF16), ([50, 0, 33], 130, 5, 2, F32),
                                              ([21, 90], 3, 33, 1, F16)])
def test_steps_as_given(lens, C, N, G, dtype):
    """Positive steps without a softplus: every value inside fp32's range."""
    d = _drop(L.scan_make(C + N + 7, lens, C, N, G, dtype, False), "dbias")
    out, final, kept = selective_scan(*_args(d), **_layer(d, False), initial_state=d["h0"],
                                      output_final_state=True, cu_seqlens=d["cu"],
                                      return_chunk_states=True)
    want = _want(d, lens, False)
    assert want.out.known.all()
    L.check("out", out, want.out, dtype)
    for i in range(len(lens)):
        L.check("final %d" % i, final[i], want.final[i], F32)
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, False), initial_state=d["h0"],
                                  dfinal_state=d["dfinal"], cu_seqlens=d["cu"], chunk_states=kept,
                                  output_dinitial_state=True)
    _check_backward(d, lens, False, dtype, got)


@pytest.mark.parametrize("T,C,N,dtype", [(3000, 192, 4, F32), (9000, 70, 2, BF16)])
def test_long_tiles(T, C, N, dtype):
    """Enough work for tiles of more than 16 tokens, in both passes."""
    d = L.scan_make(21, [T // 2 + 5, 0, T // 2 - 6, 1], C, N, 1, dtype, True)
    tiles = _check_wide(d, [T // 2 + 5, 0, T // 2 - 6, 1], C, 40, dtype)
    assert tiles < (T + 15) // 16


def _check_wide(d, lens, C, reps, dtype):
    """Both passes of a layer whose channels are `reps` times those of `d`, a group
    each time: the reference forms one group."""
    wide = {k: (d[k].repeat(1, reps) if k in ("x", "z", "delta", "dy") else
                d[k].repeat(reps, 1) if k == "A" else d[k].repeat(reps) if k in ("D", "dbias") else
                d[k].repeat(1, reps, 1) if k in ("h0", "dfinal", "B", "C") else d[k]) for k in d}
    out, final, kept = selective_scan(*_args(wide), **_layer(wide, True), initial_state=wide["h0"],
                                      output_final_state=True, cu_seqlens=d["cu"],
                                      return_chunk_states=True)
    plain = selective_scan(*_args(wide), **_layer(wide, True), initial_state=wide["h0"],
                           cu_seqlens=d["cu"])
    got = selective_scan_backward(wide["dy"], *_args(wide), **_layer(wide, True),
                                  initial_state=wide["h0"], dfinal_state=wide["dfinal"],
                                  cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)
    want = _want(d, lens, True)
    back = want.backward()
    for k in (0, 1, reps - 1):
        part = slice(k * C, (k + 1) * C)
        L.check("out", out[:, part], want.out, dtype)
        L.check("plain", plain[:, part], want.out, dtype)
        for i in range(len(lens)):
            L.check("final", final[i, part], want.final[i], F32)
        cut = {"dx": got[0][:, part], "ddelta": got[1][:, part], "dA": got[2][part],
               "dB": got[3][:, k:k + 1], "dC": got[4][:, k:k + 1], "dD": got[5][part],
               "dz": got[6][:, part], "dbias": got[7][part], "dh0": got[8][:, part]}
        for name, g in cut.items():
            L.check(name, g, back[name], F32 if name in FP32_GRADS else dtype)
    return kept.shape[0]


@pytest.mark.parametrize("lens,C,reps,N,dtype", [
    ([1000, 0, 1037, 63], 16, 520, 16, BF16), ([257, 0, 300, 1], 64, 50, 32, F32),
    ([130, 17, 253], 64, 52, 64, BF16), ([90, 500, 33], 64, 70, 8, F16)])
def test_wide_layers(lens, C, reps, N, dtype):
    """Layers whose forward pass walks along the tokens, with what it leaves for the
    backward pass."""
    d = L.scan_make(C + N + 2, lens, C, N, 1, dtype, True)
    _check_wide(d, lens, C, reps, dtype)


@pytest.mark.parametrize("lens,C,N,G,dtype", [
    ([250, 0, 300, 90, 60, 1, 16, 17], 24, 16, 1, BF16), ([13] * 50 + [0] * 5 + [7] * 10, 20, 16, 2, F32),
    ([700, 33, 800, 130], 9, 8, 1, F16), ([128, 128, 0, 256, 2], 40, 16, 1, F32), ([30, 2], 8, 64, 1, F32)])
def test_walks_of_segments(lens, C, N, G, dtype):
    """Batches that several workgroups walk along, and the same ones by tiles: B and C
    at odd addresses."""
    T, n = sum(lens), len(lens)
    d = L.scan_make(C + N + 4, lens, C, N, G, dtype, True)
    want = _want(d, lens, True)
    both = torch.empty((T, 2 * G * N + 3), device="cuda", dtype=dtype)
    odd = dict(d, B=both[:, 1:1 + G * N].view(T, G, N), C=both[:, 2 + G * N:2 + 2 * G * N].view(T, G, N))
    odd["B"].copy_(d["B"])
    odd["C"].copy_(d["C"])
    for k in (d, odd):
        idx = torch.randperm(n + 3, generator=torch.Generator().manual_seed(4))[:n].cuda()
        pool = torch.zeros((n + 3, C, N), device="cuda")
        pool[idx] = d["h0"]
        status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
        out, final = selective_scan(*_args(k), **_layer(k, True), initial_state=d["h0"],
                                    output_final_state=True, cu_seqlens=d["cu"])
        again = selective_scan(*_args(k), **_layer(k, True), initial_state=pool, output_state=pool,
                               output_final_state=True, cu_seqlens=d["cu"], state_indices=idx,
                               status=status)[0]
        L.check("out", out, want.out, dtype)
        for i in range(n):
            L.check("final %d" % i, final[i], want.final[i], F32)
        assert L.same(out, again) and L.same(pool[idx], final) and status.item() == 0


@pytest.mark.parametrize("N", [3, 70])
def test_rows_outside_every_sequence(N):
    lens = [9] * N
    d = L.scan_make(5, lens, 6, 4, 1, F32, True, tail=77)
    cu = (d["cu"] + 30).to(torch.int64)
    out = torch.full_like(d["x"], 7.0)
    selective_scan(*_args(d), **_layer(d, True), cu_seqlens=cu, output=out)
    want = _want(_drop(d, "h0"), lens, True, 30)
    span = slice(30, 30 + 9 * N)
    L.check("out", out[span], want.out[span], F32)
    assert (out[:30] == 7).all() and (out[30 + 9 * N:] == 7).all()
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, True), cu_seqlens=cu)
    _check_backward(_drop(d, "h0", "dfinal"), lens, True, F32, got, 30)
    for k in (0, 1, 3, 4, 6):
        assert not got[k][:30].any() and not got[k][30 + 9 * N:].any()


@pytest.mark.parametrize("dtype", [F32, BF16, F16, torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("n,N", [(5, 16), (66, 6)])
def test_pool_in_place(dtype, n, N):
    """States of every type in pool rows worked on in place, sequences over many
    tiles among them; rows out of range start from zero and are not written."""
    lens = [(37 * i) % 90 for i in range(n)]
    C = 10
    d = L.scan_make(8, lens, C, N, 1, F32, True)
    pool = torch.randn((n + 9, C, N), generator=torch.Generator().manual_seed(1)).cuda().to(dtype)
    before = pool.clone()
    idx = torch.randperm(n + 9, generator=torch.Generator().manual_seed(2))[:n].to(torch.int32).cuda()
    idx[1], idx[3] = -1, n + 9
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, final = selective_scan(*_args(d), **_layer(d, True), initial_state=pool,
                                output_final_state=True, cu_seqlens=d["cu"], output_state=pool,
                                state_indices=idx, status=status)
    assert final is pool and status.item() == nat.STATUS_STATE_INDEX
    rows = idx.tolist()
    d["h0"] = torch.stack([before[r].float() if 0 <= r < n + 9 else
                           torch.zeros((C, N), device="cuda") for r in rows])
    want = _want(d, lens, True)
    L.check("out", out, want.out, F32)
    for r in range(n + 9):
        if r in rows:
            L.check("row %d" % r, pool[r], want.final[rows.index(r)], dtype)
        else:
            assert torch.equal(pool[r].view(torch.uint8), before[r].view(torch.uint8))
    other = torch.zeros_like(before)  # and into another pool: the empty sequences too
    selective_scan(*_args(d), **_layer(d, True), initial_state=before, output_final_state=True,
                   cu_seqlens=d["cu"], output_state=other, state_indices=idx)
    for r in set(rows) & set(range(n + 9)):
        assert torch.equal(other[r].view(torch.uint8), pool[r].view(torch.uint8))


def test_strided_tokens():
    """Every input a slice of wider rows."""
    lens, C, N = [40, 0, 90], 70, 6
    d = L.scan_make(9, lens, C, N, 2, BF16, True)
    s = dict(d)
    for k in ("x", "delta", "z", "dy"):
        s[k] = torch.randn((130, 2 * C + 3), device="cuda").to(BF16)[:, 1:1 + C]
        s[k].copy_(d[k])
    both = torch.randn((130, 2, 2, N), device="cuda").to(BF16)
    s["B"], s["C"] = both[:, 0], both[:, 1]
    s["B"].copy_(d["B"])
    s["C"].copy_(d["C"])
    out = selective_scan(*_args(s), **_layer(s, True), cu_seqlens=d["cu"])
    L.check("out", out, _want(_drop(d, "h0"), lens, True).out, BF16)
    got = selective_scan_backward(s["dy"], *_args(s), **_layer(s, True), cu_seqlens=d["cu"])
    _check_backward(_drop(d, "h0", "dfinal"), lens, True, BF16, got)


@pytest.mark.parametrize("n,C,N,G,dtype,state", [
    (1, 1, 1, 1, F32, F32), (6, 200, 16, 2, F16, F32), (70, 33, 4, 1, BF16, BF16),
    (5, 24, 64, 1, BF16, F32), (3, 8, 32, 2, F32, torch.float8_e5m2), (4, 40, 8, 1, F32, F16),
    (4, 7, 19, 1, F32, F32)])
def test_decode(n, C, N, G, dtype, state):
    d = L.scan_make(31, [1] * n, C, N, G, dtype, True)
    pool = torch.randn((n + 2, C, N), device="cuda").to(state)
    before = pool.clone()
    idx = (torch.arange(n, device="cuda") + 1).to(torch.int64)
    out, _ = selective_scan_decode(*_args(d), **_layer(d, True), initial_state=pool,
                                   output_state=pool, state_indices=idx)
    d["h0"] = before[1:n + 1].float()
    want = _want(d, [1] * n, True)
    L.check("out", out, want.out, dtype)
    for i in range(n):
        L.check("state %d" % i, pool[1 + i], want.final[i], state)
    for r in (0, n + 1):
        assert torch.equal(pool[r].view(torch.uint8), before[r].view(torch.uint8))
    out, final = selective_scan_decode(*_args(d), delta_softplus=True)
    few = _want(_drop(d, "D", "z", "dbias", "h0"), [1] * n, True)
    L.check("plain out", out, few.out, dtype)
    for i in range(n):
        L.check("plain state", final[i], few.final[i], F32)


def test_decode_bad_rows():
    d = L.scan_make(32, [1] * 4, 48, 16)
    pool = torch.randn((3, 48, 16), device="cuda")
    before = pool.clone()
    idx = torch.tensor([2, -1, 0, 3], device="cuda", dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = selective_scan_decode(*_args(d), **_layer(d, True), initial_state=pool,
                                   output_state=pool, state_indices=idx, status=status)
    assert status.item() == nat.STATUS_STATE_INDEX
    zero = torch.zeros_like(before[0])
    d["h0"] = torch.stack([before[2], zero, before[0], zero])
    want = _want(d, [1] * 4, True)
    L.check("out", out, want.out, F32)
    L.check("row 2", pool[2], want.final[0], F32)
    L.check("row 0", pool[0], want.final[2], F32)
    assert torch.equal(pool[1], before[1])


def test_a_nan_stays_in_its_sequence_and_channel():
    lens = [30, 30, 30]
    d = L.scan_make(33, lens, 5, 4)
    d["x"][40, 2] = float("nan")
    d["h0"][2, 3, 1] = float("inf")
    out, final, kept = selective_scan(*_args(d), **_layer(d, True), initial_state=d["h0"],
                                      output_final_state=True, cu_seqlens=d["cu"],
                                      return_chunk_states=True)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[40:60, 2] = True
    want[60:90, 3] = True
    assert torch.equal(bad, want)
    assert torch.isinf(final[2, 3, 1]) and torch.isfinite(final[0]).all()
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, True), initial_state=d["h0"],
                                  cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)
    assert torch.isfinite(got[0][:30]).all() and torch.isfinite(got[8][0]).all()


def test_steps_of_zero_and_strong_decay():
    """d = 0 leaves the state as it is; a decay that underflows forgets it."""
    lens = [40, 40]
    d = L.scan_make(34, lens, 4, 4, 1, F32, False)
    d["delta"][:40] = 0.0
    d["delta"][40:] = 90.0
    d["A"].fill_(-4.0)
    out, final = selective_scan(*_args(d), initial_state=d["h0"], output_final_state=True,
                                cu_seqlens=d["cu"])
    assert torch.equal(final[0], d["h0"][0])
    last = (90.0 * d["x"][79])[:, None] * d["B"][79, 0]
    assert torch.allclose(final[1], last, rtol=3 * 2.0 ** -24, atol=0)
    assert torch.isfinite(out).all()


def _infinite(N):
    """An infinite token or step makes its channel's states infinite, and with
    coefficients above 0 and no D the outputs: infinite, not NaN."""
    lens, C = [70, 30], 6
    d = _drop(L.scan_make(38, lens, C, N, 1, F32, False), "D", "z", "dbias")
    for k in ("x", "B", "C"):
        d[k] = d[k].abs() + 0.1
    d["delta"].fill_(0.25)
    d["x"][20, 1] = d["x"][93, 4] = float("inf")
    d["delta"][40, 2] = float("inf")
    want = torch.zeros((100, C), dtype=torch.bool, device="cuda")
    want[20:70, 1] = want[93:, 4] = want[40:70, 2] = True
    out, final = selective_scan(*_args(d), initial_state=d["h0"].abs(), output_final_state=True,
                                cu_seqlens=d["cu"])
    assert torch.equal(out == float("inf"), want) and not torch.isnan(out).any()
    ends = torch.stack([want[69], want[99]])[:, :, None].expand(2, C, N)
    assert torch.equal(final == float("inf"), ends) and not torch.isnan(final).any()
    out, final = selective_scan_decode(*_args(d))
    here = torch.zeros_like(want)
    here[20, 1] = here[93, 4] = here[40, 2] = True
    assert torch.equal(out == float("inf"), here) and not torch.isnan(out).any()
    assert torch.equal(final == float("inf"), here[:, :, None].expand(100, C, N))


@pytest.mark.parametrize("N", [8, 16, 64])
def test_infinite_inputs_without_a_skip(N):
    _infinite(N)


@pytest.mark.parametrize("N", [1, 3, 12, 33])
def test_infinite_inputs_with_any_number_of_states(N):
    """Numbers of states that kernels are not compiled for."""
    _infinite(N)


@pytest.mark.parametrize("N", [4, 16])
def test_infinite_gradients_without_a_skip(N):
    """The gradient of an output of channel 1 is infinite: that of its inputs up to
    there too, not NaN."""
    lens = [40, 30]
    d = L.scan_make(39, lens, 6, N, 1, F32, False)
    for k in ("x", "B", "C"):
        d[k] = d[k].abs() + 0.1
    d["dy"][60, 1] = float("inf")
    dx = selective_scan_backward(d["dy"], *_args(d), cu_seqlens=d["cu"])[0]
    want = torch.zeros((70, 6), dtype=torch.bool, device="cuda")
    want[40:61, 1] = True
    assert torch.equal(dx == float("inf"), want) and not torch.isnan(dx).any()


def test_softplus_over_its_range():
    """Large and very small arguments keep their relative precision."""
    d = L.scan_make(35, [64], 1, 1, 1, F32, True)
    d["delta"] = torch.linspace(-80, 80, 64, device="cuda")[:, None].contiguous()
    d["A"].fill_(-1e-9)
    few = _drop(d, "D", "z", "dbias", "h0")
    final = selective_scan_decode(d["x"], d["delta"], d["A"], d["B"], d["C"], delta_softplus=True)[1]
    want = _want(few, [1] * 64, True)
    for i in range(64):
        L.check("state %d" % i, final[i], want.final[i], F32)


def test_sequence_bounds_that_are_wrong():
    d = L.scan_make(14, [20, 20], 32, 4)
    for cu in ([0, 30, 20], [0, 20, 99], [-5, 20, 40]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = selective_scan(*_args(d), cu_seqlens=torch.tensor(cu).cuda(), status=status)
        assert status.item() == nat.STATUS_CU_SEQLENS and out.shape == (40, 32)


# The walk (8, 16, 32 or 64 states in aligned rows, few enough tokens: 768 of 16 states
# where there are few channels): the same as above, over segments and over sequences
# that end where a run of 16 tokens or a step of eight runs does.

@pytest.mark.parametrize("N,dtype", [(8, F32), (16, BF16)])
def test_walks_leave_the_workspace_alone(N, dtype):
    """States before tiles are written for a caller who wants them only."""
    lens = [130, 20, 300, 0, 64, 1]
    d = L.scan_make(46, lens, 40, N, 1, dtype, True)
    ws = torch.full((1 << 24,), 7, dtype=torch.uint8, device="cuda")
    out, kept = selective_scan(*_args(d), **_layer(d, True), cu_seqlens=d["cu"], workspace=ws,
                               return_chunk_states=True)
    again = selective_scan(*_args(d), **_layer(d, True), cu_seqlens=d["cu"], workspace=ws)
    assert L.same(out, again) and (ws == 7).all()
    want = _want(_drop(d, "h0"), lens, True)
    L.check("out", out, want.out, dtype)
    tile = (sum(lens) + kept.shape[0] - 1) // kept.shape[0]
    tile = 1 << (tile - 1).bit_length()
    for k in range(1, kept.shape[0]):  # in the middle of a sequence
        i = int(np.searchsorted(np.cumsum(lens), tile * k, side="right"))
        if tile * k > sum(lens[:i]):
            L.check("tile %d" % k, kept[k].t(), want.h[tile * k - 1, i], F32)


@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("lens", [[126, 200, 128, 90, 16, 0, 60], [7] * 70])
def test_walks_leave_rows_outside_alone(lens, N):
    d = L.scan_make(40, lens, 6, N, 1, F32, True, tail=77)
    cu, T = (d["cu"] + 30).to(torch.int64), sum(lens)
    out = torch.full_like(d["x"], 7.0)
    kept = selective_scan(*_args(d), **_layer(d, True), cu_seqlens=cu, output=out,
                          return_chunk_states=True)[1]
    want = _want(_drop(d, "h0"), lens, True, 30)
    span = slice(30, 30 + T)
    L.check("out", out[span], want.out[span], F32)
    assert (out[:30] == 7).all() and (out[30 + T:] == 7).all()
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, True), cu_seqlens=cu,
                                  chunk_states=kept)
    _check_backward(_drop(d, "h0", "dfinal"), lens, True, F32, got, 30)


@pytest.mark.parametrize("N", [8, 16])
def test_walks_keep_a_nan_in_its_sequence_and_channel(N):
    lens = [128, 112, 16, 30, 40, 128, 250]
    d = L.scan_make(41, lens, 5, N)
    starts = [0] + np.cumsum(lens).tolist()
    d["x"][starts[0] + 127, 1] = float("nan")     # a step's last token
    d["delta"][starts[2] + 15, 2] = float("nan")  # a run's last token
    d["x"][starts[3] + 5, 4] = float("nan")
    d["h0"][5, 3, 1] = float("inf")
    out, final, kept = selective_scan(*_args(d), **_layer(d, True), initial_state=d["h0"],
                                      output_final_state=True, cu_seqlens=d["cu"],
                                      return_chunk_states=True)
    want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    want[127, 1] = want[starts[2] + 15, 2] = True
    want[starts[3] + 5:starts[4], 4] = True
    want[starts[5]:starts[6], 3] = True
    assert torch.equal(~torch.isfinite(out), want)
    bad = torch.zeros((7, 5), dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[2, 2] = bad[3, 4] = bad[5, 3] = True
    assert torch.equal(~torch.isfinite(final).all(2), bad)
    assert torch.isinf(final[5, 3, 1]) and torch.isnan(final[0, 1]).all()
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, True), initial_state=d["h0"],
                                  cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)
    for i in (1, 4, 6):
        assert torch.isfinite(got[0][starts[i]:starts[i + 1]]).all()
        assert torch.isfinite(got[8][i]).all()


@pytest.mark.parametrize("N", [4, 8, 16, 64])
def test_an_infinite_state_under_a_decay_that_underflows(N):
    """Every token's decay is above 0, that of a run or tile is not."""
    lens = [300, 40]
    d = L.scan_make(42, lens, 4, N, 1, F32, False)
    d["delta"].fill_(2.0)
    d["A"].fill_(-4.0)
    d["h0"][0, 2] = float("inf")
    d["h0"][1, 1] = -float("inf")
    d["C"].abs_()
    out, final = selective_scan(*_args(d), initial_state=d["h0"], output_final_state=True,
                                cu_seqlens=d["cu"])
    assert (out[:300, 2] == float("inf")).all() and (out[300:, 1] == -float("inf")).all()
    assert (final[0, 2] == float("inf")).all() and (final[1, 1] == -float("inf")).all()
    assert torch.isfinite(out[:, [0, 3]]).all() and torch.isfinite(final[:, [0, 3]]).all()


@pytest.mark.parametrize("N", [8, 16, 64])
def test_walks_of_steps_of_zero_and_strong_decay(N):
    lens = [300, 300]
    d = L.scan_make(43, lens, 4, N, 1, F32, False)
    d["delta"][:300] = 0.0
    d["delta"][300:] = 90.0
    d["A"].fill_(-4.0)
    out, final = selective_scan(*_args(d), initial_state=d["h0"], output_final_state=True,
                                cu_seqlens=d["cu"])
    assert torch.equal(final[0], d["h0"][0])
    last = (90.0 * d["x"][599])[:, None] * d["B"][599, 0]
    assert torch.allclose(final[1], last, rtol=3 * 2.0 ** -24, atol=0)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("N", [8, 16])
def test_walks_over_sequence_bounds_that_are_wrong(N):
    d = L.scan_make(44, [350, 350], 32, N)
    for cu, used in (([0, 500, 300, 650], 650), ([0, 300, 20000], 700), ([-5, 300, 600], 600),
                     ([0] + [500, 300] * 40, 500)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(d["x"], 7.0)
        selective_scan(*_args(d), delta_softplus=True, cu_seqlens=torch.tensor(cu).cuda(),
                       status=status, output=out)
        assert status.item() == nat.STATUS_CU_SEQLENS
        assert (out[used:] == 7).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("N,G,lens", [(8, 2, [240, 0, 90, 270]), (16, 1, [240, 0, 90, 270]),
                                      (64, 2, [100, 0, 60, 90])])
def test_walks_over_strided_tokens(N, G, lens):
    """Every input a slice of wider rows, B and C on boundaries of 16 bytes."""
    T, C = sum(lens), 70
    d = L.scan_make(45, lens, C, N, G, BF16, True)
    s = dict(d)
    for i, k in enumerate(("x", "delta", "z")):
        s[k] = torch.randn((T, 2 * C + 3 + i), device="cuda").to(BF16)[:, 1:1 + C]
        s[k].copy_(d[k])
    both = torch.randn((T, 3, G, N), device="cuda").to(BF16)
    s["B"], s["C"] = both[:, 0], both[:, 2]
    s["B"].copy_(d["B"])
    s["C"].copy_(d["C"])
    out, final = selective_scan(*_args(s), **_layer(s, True), initial_state=d["h0"],
                                output_final_state=True, cu_seqlens=d["cu"])
    want = _want(d, lens, True)
    L.check("out", out, want.out, BF16)
    for i in range(len(lens)):
        L.check("final %d" % i, final[i], want.final[i], F32)


@pytest.mark.parametrize("lens,N,tail", [([300, 0, 200, 12], 8, 60), ([300, 0, 200, 12], 5, 60),
                                          ([3, 9], 8, 2), ([3, 9], 5, 2), ([40] * 70, 16, 9)])
def test_all_chunk_states_are_written(lens, N, tail):
    """Also those of tiles that begin with a sequence or outside of any: zeros, not
    what the memory held."""
    d = L.scan_make(47, lens, 6, N, 1, F32, True, tail=tail)
    cu = d["cu"] + tail // 2
    rows = (sum(lens) + tail + 15) // 16
    for fill in (float("nan"), 1.0):
        old = torch.full((rows, N, 6), fill, device="cuda")
        del old  # (the next tensor of this size takes its memory)
        kept = selective_scan(*_args(d), **_layer(d, True), initial_state=d["h0"], cu_seqlens=cu,
                              return_chunk_states=True)[1]
        assert kept.shape[0] == rows and not kept[0].any()
        if fill != fill:
            first = kept
    assert L.same(kept, first) and torch.isfinite(kept).all()


def test_no_tokens():
    d = L.scan_make(36, [0, 0], 8, 4)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    out, final = selective_scan(*_args(d), **_layer(d, True), initial_state=d["h0"],
                                output_final_state=True, cu_seqlens=d["cu"], status=status)
    assert out.shape == (0, 8) and torch.equal(final, d["h0"]) and status.item() == 0
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, True), initial_state=d["h0"],
                                  dfinal_state=d["dfinal"], cu_seqlens=d["cu"],
                                  output_dinitial_state=True)
    assert torch.equal(got[8], d["dfinal"])
    for k in (2, 5, 7):
        assert not got[k].any()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, final = selective_scan(*_args(d), output_final_state=True, cu_seqlens=none)
    assert final.shape == (0, 8, 4)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd(dtype):
    lens = [12, 0, 2, 50]
    d = L.scan_make(16, lens, 10, 8, 2, dtype, True)
    names = ("x", "delta", "A", "B", "C", "D", "z", "dbias", "h0")
    leaf = {k: d[k].detach().clone().requires_grad_() for k in names}
    out, final = selective_scan(*_args(leaf), **_layer(leaf, True), initial_state=leaf["h0"],
                                output_final_state=True, cu_seqlens=d["cu"])
    torch.autograd.backward([out, final], [d["dy"], d["dfinal"]])
    _check_backward(d, lens, True, dtype, [leaf[k].grad for k in names])
    # only some of them
    x = d["x"].clone().requires_grad_()
    selective_scan(x, *_args(d)[1:], delta_softplus=True, cu_seqlens=d["cu"]).backward(d["dy"])
    L.check("dx", x.grad, _want(_drop(d, "D", "z", "dbias", "h0", "dfinal"), lens, True).backward()["dx"],
            dtype)


def test_gradients_against_differences():
    lens = [9, 2, 30]
    d = L.scan_make(17, lens, 3, 2, 1, F32, True)
    got = selective_scan_backward(d["dy"], *_args(d), **_layer(d, True), initial_state=d["h0"],
                                  dfinal_state=d["dfinal"], cu_seqlens=d["cu"],
                                  output_dinitial_state=True)
    n = {k: f64(v) for k, v in d.items() if k != "cu"}
    bound = L.Scan(n, lens, True).backward()

    def loss(**at):
        s = L.Scan(dict(n, **at), lens, True)
        return (s.out.v * n["dy"]).sum() + sum((f.v * g).sum() for f, g in zip(s.final, n["dfinal"]))

    rng = np.random.default_rng(0)
    for k, g, grad in zip(("x", "delta", "A", "B", "C", "D", "z", "dbias", "h0"), GRADS, got):
        way = rng.standard_normal(n[k].shape)
        h = 1e-5
        slope = (loss(**{k: n[k] + h * way}) - loss(**{k: n[k] - h * way})) / (2 * h)
        # the gradient's own bound, and 1e-7 for what the difference leaves (h^2 and
        # 2^-53 / h of the loss)
        lim = (np.abs(way) * bound[g].e).sum() + 1e-7 * (1 + np.abs(f64(grad) * way).sum())
        assert abs(slope - (f64(grad) * way).sum()) <= lim, k


def test_refusals_on_the_device():
    d = L.scan_make(18, [8], 16, 4)
    x, delta, A, B, C = _args(d)
    scan = lambda *a, **k: (lambda: selective_scan(*a, **k))  # noqa: E731
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = [
        scan(x, delta[:4], A, B, C), scan(x, delta.to(BF16), A, B, C), scan(x, delta, A.to(BF16), B, C),
        scan(x, delta, A.t(), B, C), scan(x, delta, A, B[:, :, :3], C), scan(x, delta, A, B, C.to(F16)),
        scan(x, delta, torch.zeros((16, 65), device="cuda"), B, C),
        scan(x, delta, A, B.expand(8, 3, 4).contiguous(), C.expand(8, 3, 4).contiguous()),
        scan(x, delta, A, B, C, D=d["D"][:3]), scan(x, delta, A, B, C, output=x),
        scan(x, delta, A, B, C, z=x, output=x), scan(x, delta, A, B, C, initial_state=d["h0"][:, :3]),
        scan(x, delta, A, B, C, state_indices=one), scan(x.t(), delta, A, B, C),
        scan(x, delta, A.clone().requires_grad_(), B, C, status=one),
        lambda: selective_scan_backward(d["dy"], x, delta, A, B, C, initial_state=d["h0"].to(BF16)),
        lambda: selective_scan_backward(d["dy"], x, delta, A, B, C, chunk_states=d["h0"]),
        lambda: selective_scan_decode(x, delta, A, B, C, initial_state=d["h0"]),
        lambda: selective_scan_decode(x, delta, A.clone().requires_grad_(), B, C),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
