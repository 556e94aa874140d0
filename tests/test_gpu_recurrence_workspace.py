"""GPU tests of the recurrence's workspace: waits of the chain that end whatever
the workspace holds, and calls that share one against the rules."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    _native as nat, gated_linear_recurrence, gated_linear_recurrence_backward)
from tests import recurrence_testlib as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.fixture
def wait_limit():
    """The number of looks after which a wait of the chain gives up."""
    limit = ctypes.c_uint32.in_dll(nat.lib(), "_ZN3gdn14rec_wait_limitE")
    before = limit.value
    assert before >= 1 << 16
    yield limit
    torch.cuda.synchronize()
    limit.value = before


def _step(d, workspace=None):
    out, fin, kept = gated_linear_recurrence(
        d["x"], d["g"], initial_state=d["h0"], output_final_state=True, cu_seqlens=d["cu"],
        return_chunk_states=True, workspace=workspace)
    return (out, fin) + gated_linear_recurrence_backward(
        d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True, workspace=workspace)


@pytest.mark.parametrize("looks", [0, 3])
@pytest.mark.parametrize("dtype,per_head", [(torch.float32, False), (torch.bfloat16, True)])
def test_waits_that_give_up(wait_limit, looks, dtype, per_head):
    """A wait that gives up leaves NaN behind it up to the next sequence; what
    did not wait for it is right, and so is the next call."""
    d = R.make(70, [5000, 0, 3, 2500], 4, 64, dtype, torch.float32, per_head)
    want = _step(d)
    torch.cuda.synchronize()
    wait_limit.value = looks
    got = _step(d)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert ((g == w) | torch.isnan(g)).all()
    wait_limit.value = 1 << 20
    for w, g in zip(want, _step(d)):
        assert torch.equal(w, g)


def test_calls_on_two_streams_with_one_workspace_end(wait_limit):
    """Against the rules, and wrong; but the calls end, and write only their
    own rows."""
    ds = [R.make(71, [3000, 500], 4, 64, torch.bfloat16),
          R.make(72, [17] * 120, 4, 64, torch.bfloat16)]
    want = [_step(d) for d in ds]
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    bufs = []
    for d in ds:
        T = d["x"].shape[0]
        bufs.append(torch.full((T + 400, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    wait_limit.value = 200
    for _ in range(10):
        for d, buf, s in zip(ds, bufs, streams):
            T = d["x"].shape[0]
            with torch.cuda.stream(s):
                gated_linear_recurrence(d["x"], d["g"], initial_state=d["h0"],
                                        cu_seqlens=d["cu"], output=buf[200:200 + T], workspace=ws)
    torch.cuda.synchronize()
    for buf in bufs:
        assert (buf[:200] == 7).all() and (buf[-200:] == 7).all()
    wait_limit.value = 1 << 20
    for d, w in zip(ds, want):
        for a, b in zip(w, _step(d, ws)):
            assert torch.equal(a, b)
