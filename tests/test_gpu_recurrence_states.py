"""GPU tests of the backward pass that forms its states itself, where its scan and
the forward one are cut into different tiles: 16-bit x with head gates."""
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


@pytest.mark.parametrize("lens", [[1], [64], [65], [100], [128], [129], [700, 3, 0, 129],
                                  [5] * 13 + [0] * 60, [30, 0, 2] * 40, [9000]])
@pytest.mark.parametrize("dtype,gate", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("H,D", [(3, 32), (5, 64), (2, 128)])
def test_head_gates_without_kept_states(lens, dtype, gate, H, D):
    d = R.make(95, lens, H, D, dtype, gate, per_head=True)
    kw = dict(initial_state=d["h0"], cu_seqlens=d["cu"])
    out, fin, kept = gated_linear_recurrence(d["x"], d["g"], output_final_state=True,
                                             return_chunk_states=True, **kw)
    kw.update(dfinal_state=d["dfinal"], output_dinitial_state=True)
    want = gated_linear_recurrence_backward(d["dy"], d["x"], d["g"], chunk_states=kept, **kw)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = gated_linear_recurrence_backward(d["dy"], d["x"], d["g"], status=st, **kw)
    assert st.item() == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    w = R.backward(R.f64(d["dy"]), R.f64(d["x"]), R.f64(d["g"]), lens, R.f64(d["h0"]),
                   R.f64(d["dfinal"]))
    for name, g in zip(("dx", "dg", "dh0"), got):
        R.check(name, g, *w[name], g.dtype)
