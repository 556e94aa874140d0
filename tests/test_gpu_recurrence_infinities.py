"""GPU tests of infinite states over long runs of strong gates, against the
definition followed token by token: an infinity stays under gates above 0 however
small their product, becomes NaN under a gate of 0, and stays in its sequence."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    gated_linear_recurrence, gated_linear_recurrence_backward)
from tests import recurrence_testlib as R  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _definition(d, lens):
    """h, final, dx, dg, dh0 in fp64 (infinities and NaN as they come)."""
    x, g, dy, h0, dfin = (R.f64(d[k]) for k in ("x", "g", "dy", "h0", "dfinal"))
    gw = R.wide(g, x.shape)
    h, dx, dg = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    final, dh0 = h0.copy(), dfin.copy()
    t0 = 0
    with np.errstate(invalid="ignore", over="ignore"):
        for i, n in enumerate(lens):
            s = h0[i]
            for t in range(t0, t0 + n):
                s = gw[t] * s + x[t]
                h[t] = s
            final[i] = s
            k = dfin[i]
            for t in range(t0 + n - 1, t0 - 1, -1):
                dx[t] = dy[t] + k
                dg[t] = dx[t] * (h[t - 1] if t > t0 else h0[i])
                k = gw[t] * dx[t]
            dh0[i] = k
            t0 += n
        if g.ndim == 2:
            dg = dg.sum(-1)
    return h, final, dx, dg, dh0


def _same_kind(name, got, want):
    """NaN where NaN, an infinity of the same sign where infinite, else finite."""
    got = R.f64(got)
    for kind, f in (("nan", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
        bad = f(got) != f(want)
        assert not bad.any(), (name, kind, np.argwhere(bad)[:3].tolist(), int(bad.sum()))


def _run(d):
    out, fin, kept = gated_linear_recurrence(
        d["x"], d["g"], initial_state=d["h0"], output_final_state=True, cu_seqlens=d["cu"],
        return_chunk_states=True)
    return (out, fin) + gated_linear_recurrence_backward(
        d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)


# tiles of 64 or 128 tokens, groups of 8 tiles, windows of 8 groups
@pytest.mark.parametrize("lens", [[60], [300, 0, 700], [9000], [5000, 4000]])
@pytest.mark.parametrize("gate", [0.5, 0.25, 1e-3, 1e-6])
@pytest.mark.parametrize("dtype,gtype,per_head", [
    (F32, F32, False), (F32, F32, True), (BF16, F32, False), (BF16, BF16, True),
    (F16, F16, False)])
def test_infinity_under_strong_gates(lens, gate, dtype, gtype, per_head):
    d = R.make(90, lens, 2, 32, dtype, gtype, per_head)
    shape = d["g"].shape
    scale = torch.rand(shape, generator=torch.Generator().manual_seed(91)).cuda() + 0.5
    d["g"] = (gate * scale).clamp(min=1e-7).to(gtype)
    assert (d["g"] > 0).all()
    T = sum(lens)
    d["x"][5, 0, 1] = float("inf")
    d["x"][T // 3, 1, 7] = -float("inf")
    d["h0"][-1, 1, 3] = float("inf")
    d["dy"][T - 4, 0, 2] = -float("inf")
    d["dy"][2 * T // 3, 1, 9] = float("inf")
    d["dfinal"][0, 0, 4] = float("inf")
    d["dfinal"][-1, 1, 30] = -float("inf")
    # a gate of 0 behind an infinity
    d["x"][10, 1, 11] = float("inf")
    if per_head:
        d["x"][10, 1, 11] = 1.0
    else:
        d["g"][T // 2, 1, 11] = 0.0
    want = _definition(d, lens)
    for name, got, w in zip(("out", "final", "dx", "dg", "dh0"), _run(d), want):
        if name == "dg" and per_head:
            # a sum of terms: infinite or NaN where one of them is
            assert np.array_equal(np.isfinite(R.f64(got)), np.isfinite(w))
            continue
        _same_kind(name, got, w)


def test_zero_gates_still_end_a_state():
    """A gate of exactly 0 somewhere in a long run: nothing of the state before
    comes through, whatever the other gates' product."""
    for tokens in (100, 3000, 9000):
        d = R.make(92, [tokens], 2, 32)
        d["g"] = torch.full_like(d["g"], 1e-4)
        d["g"][20] = 0.0
        d["x"].zero_()
        d["h0"].fill_(3e38)
        out, fin = gated_linear_recurrence(d["x"], d["g"], initial_state=d["h0"],
                                           output_final_state=True, cu_seqlens=d["cu"])
        assert (out[20:] == 0).all() and (fin == 0).all()
        # and without one, what is left of it is less than the smallest normal
        d["g"][20] = 1e-4
        out = gated_linear_recurrence(d["x"], d["g"], initial_state=d["h0"], cu_seqlens=d["cu"])
        assert (out[40:].abs() <= 2.0 ** -149 * 3e38).all()
