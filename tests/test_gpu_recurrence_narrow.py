"""GPU tests of the recurrence over few channels, where most lanes of a wave have
none, and sequences that start and end at every token of a wave: states go from
and to the rows of their own sequences."""
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


LENS = {
    "two": [3, 27],
    "steps": list(range(1, 17)),
    "steps many": list(range(1, 13)) * 8,
    "pairs": [7, 9] * 9 + [16, 15, 17, 1, 31, 33],
    "long": [881, 663, 394, 1634, 428],
    "ragged": [130, 0, 20, 0, 300, 64, 1] * 3,
}
WIDTHS = [(1, 1), (1, 3), (1, 7), (1, 28), (5, 7), (1, 300)]
HEADS = [(1, 32), (3, 32), (1, 64), (1, 128), (9, 32)]


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype,gate,per_head,shape", [
    (d, g, p, s) for d, g in ((BF16, BF16), (BF16, F32), (F16, F16), (F32, F32))
    for p, shapes in ((False, WIDTHS), (True, HEADS)) for s in shapes])
def test_few_channels(lens, dtype, gate, per_head, shape):
    lens = LENS[lens]
    d = R.make(101, lens, *shape, dtype, gate, per_head)
    N, rows = len(lens), len(lens) + 6
    gen = torch.Generator().manual_seed(102)
    idx = (3 + torch.randperm(N, generator=gen)).to(torch.int32).cuda()
    pool = torch.randn((rows,) + shape, generator=gen).cuda()
    pool[idx.long()] = d["h0"]
    before = pool.clone()
    out, _, kept = gated_linear_recurrence(
        d["x"], d["g"], initial_state=pool, output_final_state=True, cu_seqlens=d["cu"],
        output_state=pool, state_indices=idx, return_chunk_states=True)
    x, g, h0 = R.f64(d["x"]), R.f64(d["g"]), R.f64(d["h0"])
    h, err, final, ferr = R.forward(x, g, lens, h0)
    R.check("out", out, h, err, dtype)
    R.check("final", pool[idx.long()], final, ferr, F32)
    assert torch.equal(pool[:3], before[:3]) and torch.equal(pool[-3:], before[-3:])
    got = gated_linear_recurrence_backward(
        d["dy"], d["x"], d["g"], initial_state=d["h0"], dfinal_state=d["dfinal"],
        cu_seqlens=d["cu"], chunk_states=kept, output_dinitial_state=True)
    want = R.backward(R.f64(d["dy"]), x, g, lens, h0, R.f64(d["dfinal"]))
    for name, t in zip(("dx", "dg", "dh0"), got):
        R.check(name, t, *want[name], t.dtype)
