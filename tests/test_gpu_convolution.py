"""GPU tests of the short causal convolution against its definition in fp64: bounds
of sequences, states, pools, strides, types, gradients, decode steps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    _native as nat, short_convolution, short_convolution_backward, short_convolution_decode)
from tests import layers_testlib as L  # noqa: E402
from tests.recurrence_testlib import f64  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _check(d, lens, act, bias=True, h0=True, begin=0, out=None, final=None):
    want, fin, _, _ = L.conv_forward(f64(d["x"]), f64(d["w"]), f64(d["bias"]) if bias else None, lens,
                                     f64(d["h0"]) if h0 else None, act, begin)
    for i, t, n in L._starts(lens, begin):
        L.check("sequence %d" % i, out[t:t + n], want[i], d["x"].dtype)
        if final is not None:
            assert np.array_equal(f64(final[i]), fin[i]), i


CASES = [
    ([1], 1, 4, F32, F32), ([0], 5, 3, F32, F32), ([2, 0, 1, 3, 4, 0], 7, 4, F32, F32),
    ([70, 1, 0, 64, 130], 64, 4, BF16, BF16), ([5, 3, 2, 1, 90], 520, 4, BF16, F32),
    ([33, 64, 31, 1, 2], 264, 3, F16, F16), ([300], 72, 2, F16, F32), ([1] * 63, 16, 4, F32, F32),
    ([3] * 64, 24, 4, BF16, BF16), ([0, 2, 7] * 40, 8, 4, F32, F32), ([65] * 70, 10, 3, BF16, F32),
    ([1000, 17, 2000], 513, 4, BF16, BF16),
]


@pytest.mark.parametrize("lens,C,W,dtype,wtype", CASES)
@pytest.mark.parametrize("act", [None, "silu"])
def test_forward(lens, C, W, dtype, wtype, act):
    d = L.conv_make(len(lens) + C, lens, C, W, dtype, wtype)
    out, final = short_convolution(d["x"], d["w"], d["bias"], act, initial_state=d["h0"],
                                   output_final_state=True, cu_seqlens=d["cu"])
    _check(d, lens, act, out=out, final=final)
    out = short_convolution(d["x"], d["w"], None, act, cu_seqlens=d["cu"])
    _check(d, lens, act, bias=False, h0=False, out=out)


@pytest.mark.parametrize("lens,C,W,dtype,wtype", CASES)
@pytest.mark.parametrize("act", [None, "silu"])
def test_backward(lens, C, W, dtype, wtype, act):
    d = L.conv_make(3 * len(lens) + C, lens, C, W, dtype, wtype)
    dx, dw, db, dh0 = short_convolution_backward(
        d["dy"], d["x"], d["w"], d["bias"], act, initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], output_dinitial_state=True)
    want = L.conv_backward(f64(d["dy"]), f64(d["x"]), f64(d["w"]), f64(d["bias"]), lens, f64(d["h0"]),
                           f64(d["dfinal"]), act)
    L.check("dx", dx, want["dx"], dtype)
    L.check("dw", dw, want["dw"], F32)
    L.check("dbias", db, want["dbias"], F32)
    L.check("dh0", dh0, want["dh0"], F32)
    again = short_convolution_backward(
        d["dy"], d["x"], d["w"], d["bias"], act, initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], output_dinitial_state=True)
    for a, b in zip((dx, dw, db, dh0), again):
        assert torch.equal(a, b)
    dx, dw, db = short_convolution_backward(d["dy"], d["x"], d["w"], None, act, cu_seqlens=d["cu"])
    want = L.conv_backward(f64(d["dy"]), f64(d["x"]), f64(d["w"]), None, lens, None, None, act)
    assert db is None
    L.check("dx", dx, want["dx"], dtype)
    L.check("dw", dw, want["dw"], F32)


@pytest.mark.parametrize("N", [3, 70])
def test_rows_outside_every_sequence(N):
    lens = [9] * N
    d = L.conv_make(5, lens, 40, 4, BF16, F32, tail=77)
    cu = (d["cu"] + 30).to(torch.int64)
    out = torch.full_like(d["x"], 7.0)
    short_convolution(d["x"], d["w"], d["bias"], "silu", cu_seqlens=cu, output=out)
    _check(d, lens, "silu", h0=False, begin=30, out=out)
    assert (out[:30] == 7).all() and (out[30 + 9 * N:] == 7).all()
    dx, dw, db = short_convolution_backward(d["dy"], d["x"], d["w"], d["bias"], "silu", cu_seqlens=cu)
    want = L.conv_backward(f64(d["dy"]), f64(d["x"]), f64(d["w"]), f64(d["bias"]), lens, None, None,
                           "silu", 30)
    L.check("dx", dx, want["dx"], BF16)
    L.check("dw", dw, want["dw"], F32)
    assert not dx[:30].any() and not dx[30 + 9 * N:].any()


@pytest.mark.parametrize("dtype", [F32, BF16, F16, torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("N", [5, 66])
def test_pool_in_place(dtype, N):
    """States of every type in pool rows worked on in place; row -1 and one out of
    range start from zero and are not written."""
    lens = [(7 * i) % 11 for i in range(N)]
    C, W = 24, 4
    d = L.conv_make(8, lens, C, W, BF16, F32)
    pool = torch.randn((N + 9, W - 1, C), generator=torch.Generator().manual_seed(1)).cuda().to(dtype)
    before = pool.clone()
    idx = torch.randperm(N + 9, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32).cuda()
    idx[1], idx[3] = -1, N + 9
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, final = short_convolution(d["x"], d["w"], d["bias"], "silu", initial_state=pool,
                                   output_final_state=True, cu_seqlens=d["cu"], output_state=pool,
                                   state_indices=idx, status=status)
    assert final is pool and status.item() == nat.STATUS_STATE_INDEX
    d["h0"] = torch.stack([before[r].float() if 0 <= r < N + 9 else torch.zeros_like(before[0]).float()
                           for r in idx.tolist()])
    _check(d, lens, "silu", out=out)
    _, fin, _, _ = L.conv_forward(f64(d["x"]), f64(d["w"]), None, lens, f64(d["h0"]), False)
    rows = idx.tolist()
    for r in range(N + 9):
        if r in rows:
            want = torch.tensor(fin[rows.index(r)]).float().to(dtype)
            assert np.array_equal(f64(pool[r]), f64(want)), r
        else:
            assert torch.equal(pool[r].view(torch.uint8), before[r].view(torch.uint8))


@pytest.mark.parametrize("dtype,C,off", [(BF16, 128, 0), (BF16, 128, 3), (F32, 36, 1), (F16, 33, 8)])
def test_strided_tokens(dtype, C, off):
    """x and dy as slices of wider rows, aligned and not."""
    lens = [40, 0, 90]
    d = L.conv_make(9, lens, C, 4, dtype, F32)
    wide = torch.randn((130, 3 * C + 8), device="cuda").to(dtype)
    for k in ("x", "dy"):
        v = wide.clone()[:, off:off + C]
        v.copy_(d[k])
        d[k] = v
    out = short_convolution(d["x"], d["w"], d["bias"], "silu", cu_seqlens=d["cu"])
    _check(d, lens, "silu", h0=False, out=out)
    dx, dw, _ = short_convolution_backward(d["dy"], d["x"], d["w"], d["bias"], "silu",
                                           cu_seqlens=d["cu"])
    want = L.conv_backward(f64(d["dy"]), f64(d["x"]), f64(d["w"]), f64(d["bias"]), lens, None, None,
                           "silu")
    L.check("dx", dx, want["dx"], dtype)
    L.check("dw", dw, want["dw"], F32)


@pytest.mark.parametrize("N,C,W,dtype,state", [(1, 1, 4, F32, F32), (6, 2048, 4, BF16, BF16),
                                               (70, 33, 3, F16, F32), (9, 72, 2, BF16, F16),
                                               (5, 64, 4, F32, torch.float8_e4m3fn)])
def test_decode_continues_the_forward_pass(N, C, W, dtype, state):
    """A prompt and three decode steps against the prompt with three tokens more."""
    lens = [i % 5 for i in range(N)]
    d = L.conv_make(12, [n + 3 for n in lens], C, W, dtype, F32)
    starts = np.concatenate([[0], np.cumsum([n + 3 for n in lens])])
    head = torch.cat([d["x"][s:s + n] for s, n in zip(starts, lens)])
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    pool = torch.zeros((N + 2, W - 1, C), device="cuda", dtype=F32).to(state)
    idx = (torch.arange(N, device="cuda") + 1).to(torch.int64)
    rows = [torch.zeros((W - 1, C)) for _ in lens]
    if head.shape[0]:
        short_convolution(head, d["w"], d["bias"], "silu", output_final_state=True, cu_seqlens=cu,
                          initial_state=pool, output_state=pool, state_indices=idx)
    narrow = lambda t: f64(t.float().to(state))  # noqa: E731
    for i, n in enumerate(lens):
        both = torch.cat([rows[i], d["x"][starts[i]:starts[i] + n].float().cpu()])
        rows[i] = torch.tensor(narrow(both[n:]))
        assert np.array_equal(f64(pool[1 + i]), rows[i].numpy())
    for k in range(3):
        x = torch.stack([d["x"][s + n + k] for s, n in zip(starts, lens)])
        out, _ = short_convolution_decode(x, d["w"], d["bias"], "silu", initial_state=pool,
                                          output_state=pool, state_indices=idx)
        want, fin, _, _ = L.conv_forward(f64(x), f64(d["w"]), f64(d["bias"]), [1] * N,
                                         np.stack([r.numpy() for r in rows]), "silu")
        L.check("step %d" % k, out, L.E(np.concatenate([w.v for w in want]),
                                        np.concatenate([w.e for w in want])), dtype)
        rows = [torch.tensor(narrow(torch.tensor(f).float())) for f in fin]
        for i in range(N):
            assert np.array_equal(f64(pool[1 + i]), rows[i].numpy())
    assert not pool[0].float().any() and not pool[N + 1].float().any()


def test_decode_in_place_and_bad_rows():
    d = L.conv_make(13, [1] * 4, 48, 4, BF16, F32)
    pool = torch.randn((3, 3, 48), device="cuda")
    before, x = pool.clone(), d["x"].clone()
    idx = torch.tensor([2, -1, 0, 3], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = short_convolution_decode(x, d["w"], None, None, initial_state=pool, output=x,
                                      output_state=pool, state_indices=idx, status=status)
    assert out is x and status.item() == nat.STATUS_STATE_INDEX
    h0 = np.stack([f64(before[2]), np.zeros((3, 48)), f64(before[0]), np.zeros((3, 48))])
    want, fin, _, _ = L.conv_forward(f64(d["x"]), f64(d["w"]), None, [1] * 4, h0, None)
    for i in range(4):
        L.check("row %d" % i, out[i:i + 1], want[i], BF16)
    assert np.array_equal(f64(pool[2]), fin[0]) and np.array_equal(f64(pool[0]), fin[2])
    assert torch.equal(pool[1], before[1])


def test_sequence_bounds_that_are_wrong():
    """Offsets that fall or leave the tokens: a status bit, nothing else is written."""
    d = L.conv_make(14, [20, 20], 32, 4, F32)
    for cu in ([0, 30, 20], [0, 20, 99], [-5, 20, 40]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = short_convolution(d["x"], d["w"], cu_seqlens=torch.tensor(cu).cuda(), status=status)
        assert status.item() == nat.STATUS_CU_SEQLENS and out.shape == (40, 32)


def test_a_nan_stays_in_its_sequence():
    lens = [10, 10, 10]
    d = L.conv_make(15, lens, 16, 4, F32)
    d["x"][15] = float("nan")
    d["h0"][2] = float("inf")
    out = short_convolution(d["x"], d["w"], d["bias"], None, initial_state=d["h0"], cu_seqlens=d["cu"])
    bad = ~torch.isfinite(out).all(1)
    assert bad.nonzero()[:, 0].tolist() == [15, 16, 17, 18, 20, 21, 22]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd(dtype):
    lens = [12, 0, 2, 50]
    d = L.conv_make(16, lens, 40, 4, dtype, dtype)
    leaves = [d[k].to(dtype).requires_grad_() for k in ("x", "w", "bias", "h0")]
    out, final = short_convolution(leaves[0], leaves[1], leaves[2], "silu", initial_state=leaves[3],
                                   output_final_state=True, cu_seqlens=d["cu"])
    torch.autograd.backward([out, final], [d["dy"], d["dfinal"]])
    want = L.conv_backward(f64(d["dy"]), f64(d["x"]), f64(d["w"]), f64(d["bias"]), lens,
                           f64(d["h0"].to(dtype)), f64(d["dfinal"]), "silu")
    for leaf, k in zip(leaves, ("dx", "dw", "dbias", "dh0")):
        assert leaf.grad.dtype == dtype
        L.check(k, leaf.grad, want[k], dtype)


def test_gradients_against_differences():
    """Differences of the definition in fp64 along a direction for each input."""
    lens, C, W = [9, 2, 30], 6, 4
    d = L.conv_make(17, lens, C, W, F32)
    dx, dw, db, dh0 = short_convolution_backward(
        d["dy"], d["x"], d["w"], d["bias"], "silu", initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], output_dinitial_state=True)
    n = {k: f64(v) for k, v in d.items()}
    bound = L.conv_backward(n["dy"], n["x"], n["w"], n["bias"], lens, n["h0"], n["dfinal"], "silu")

    def loss(**at):
        p = dict(n, **at)
        out, fin, _, _ = L.conv_forward(p["x"], p["w"], p["bias"], lens, p["h0"], "silu")
        return sum((o.v * n["dy"][t:t + k]).sum() for o, (_, t, k) in zip(out, L._starts(lens, 0))) + \
            sum((f * g).sum() for f, g in zip(fin, n["dfinal"]))

    rng = np.random.default_rng(0)
    for k, g, grad in (("x", "dx", dx), ("w", "dw", dw), ("bias", "dbias", db), ("h0", "dh0", dh0)):
        way = rng.standard_normal(n[k].shape)
        h = 1e-5
        slope = (loss(**{k: n[k] + h * way}) - loss(**{k: n[k] - h * way})) / (2 * h)
        # the gradient's own bound, and 1e-7 for what the difference leaves (h^2 and
        # 2^-53 / h of the loss)
        lim = (np.abs(way) * bound[g].e).sum() + 1e-7 * (1 + np.abs(f64(grad) * way).sum())
        assert abs(slope - (f64(grad) * way).sum()) <= lim


def test_refusals_on_the_device():
    d = L.conv_make(18, [8], 16, 4, F32)
    x, w = d["x"], d["w"]
    bad = [
        lambda: short_convolution(x, w, activation="relu"),
        lambda: short_convolution(x, w[:, :1].contiguous()),
        lambda: short_convolution(x, w.to(BF16)),
        lambda: short_convolution(x, w.t()),
        lambda: short_convolution(x, w, d["bias"].to(BF16)),
        lambda: short_convolution(x, w, output=x),
        lambda: short_convolution(x.t(), w),
        lambda: short_convolution(x, w, initial_state=d["h0"][:, :2]),
        lambda: short_convolution(x, w, state_indices=torch.zeros(1, dtype=torch.int32, device="cuda")),
        lambda: short_convolution_backward(d["dy"], x, w, dx=x),
        lambda: short_convolution_backward(d["dy"].to(BF16), x, w),
        lambda: short_convolution_decode(x, w, initial_state=d["h0"]),
        lambda: short_convolution(x, w.clone().requires_grad_(), output=torch.empty_like(x)),
        lambda: short_convolution_decode(x, w.clone().requires_grad_()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_a_gradient_buffer_without_its_input():
    """A buffer that no gradient would be written to is refused, not dropped."""
    d = L.conv_make(19, [8], 16, 4, F32)
    db = torch.full((16,), 3.0, device="cuda")
    with pytest.raises(ValueError, match="dbias"):
        short_convolution_backward(d["dy"], d["x"], d["w"], dbias=db)
    assert (db == 3).all()
    assert short_convolution_backward(d["dy"], d["x"], d["w"], d["bias"], dbias=db)[2] is db
