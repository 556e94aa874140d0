"""GPU tests of the state-pool operators' lists: rows kept and forked in one list,
conflicts by the rule, against a plain copy of the rule."""
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import state_pool_compact, state_pool_copy  # noqa: E402

pytestmark = pytest.mark.gpu

OUT, DUP, OVER = 16, 32, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _rows(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _copy_rule(pool, src, dst):
    """The pool and the status bits after a copy inside it, entry by entry."""
    n = pool.shape[0]
    want, bits = pool.clone(), 0
    ok = [s >= 0 and d >= 0 and s < n and d < n for s, d in zip(src, dst)]
    if any(v >= n or v < -1 for v in list(src) + list(dst)):
        bits |= OUT
    entries = [(i, s, d) for i, (s, d) in enumerate(zip(src, dst)) if ok[i]]
    for i, s, d in entries:
        later = any(j > i and e == d for j, _, e in entries)
        changed = s != d and any(j != i and e == s and f != e for j, f, e in entries)
        bits |= (DUP if later else 0) | (OVER if changed else 0)
        if not later and not changed:
            want[d] = pool[s]
    return want, bits


# long rows go one entry at a time, short ones in groups once there are many
@pytest.mark.parametrize("rows,row", [(16, (64, 128)), (4000, (4,)), (4000, (3,))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_kept_and_forked(rows, row, dtype):
    gen = torch.Generator().manual_seed(rows)
    ref = torch.randn((rows,) + row, generator=gen).to(dtype).cuda()
    lists = [([0, 0], [0, 1]), ([0, 0], [1, 0]), ([3, 5, 3, 5, 3], [3, 5, 6, 7, 8]),
             # a row kept and overwritten by an earlier or a later entry
             ([2, 0, 0], [0, 0, 1]), ([0, 2, 0], [0, 0, 1]),
             ([1, 0], [0, 1]), ([4, 4], [4, 4])]
    if rows > 1000:  # each of the first half kept, and forked into the second half
        half = list(range(rows // 2))
        lists.append((half + half, half + [rows // 2 + r for r in half]))
        mix = torch.randint(-2, rows + 2, (2, 3000), generator=gen).tolist()
        mix[0][::7] = mix[1][::7]  # kept rows among them
        lists.append((mix[0], mix[1]))
    for src, dst in lists:
        want, bits = _copy_rule(ref.cpu(), src, dst)
        for status in (None, _rows([-1])):
            pool = ref.clone()
            state_pool_copy(pool, _rows(src), _rows(dst), status=status)
            assert torch.equal(pool.cpu(), want), (src[:8], dst[:8])
            assert status is None or status.item() == bits


def test_compact_moves_all_pools_or_none():
    first = torch.arange(12, device="cuda", dtype=torch.float32).view(12, 1).repeat(1, 8)
    want = first.clone()
    base = torch.zeros(400, device="cuda")
    overlapping = base.as_strided((12, 8), (4, 1))  # rows that share elements
    out, where = _rows([-5, -5]), _rows([-5] * 12)
    for bad in (overlapping, base[:12].view(12, 1).expand(12, 8), first.double(), first[:11],
                first.cpu()):
        with pytest.raises(ValueError):
            state_pool_compact([first, bad], _rows([11, 7]), output_indices=out, row_map=where)
        assert torch.equal(first, want)
        assert (out == -5).all() and (where == -5).all()
    ren, n = state_pool_compact([first, want.clone()], _rows([11, 7]), output_indices=out)
    assert ren.tolist() == [1, 0] and n.item() == 2
    assert first[:2, 0].tolist() == [7, 11]


@pytest.mark.parametrize("row", [(4, 128, 128), (16, 128), (5, 7), (1,), (2, 4100)])
@pytest.mark.parametrize("frm,to", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                    (torch.float32, torch.bfloat16),
                                    (torch.bfloat16, torch.bfloat16)])
def test_pools_of_one_row(row, frm, to):
    """One checkpoint forked into a pool, and a row brought into a pool of one,
    at aligned and unaligned places."""
    gen = torch.Generator().manual_seed(1)
    n = 1
    for e in row:
        n *= e
    for off in (0, 1):
        store = torch.randn(n + off, generator=gen).to(frm).cuda()
        one = store[off:].view((1,) + row)
        pool = torch.randn((6,) + row, generator=gen).to(to).cuda()
        want = pool.clone()
        want[[1, 4]] = one[0].to(to)
        state_pool_copy(pool, _rows([0, 0]), _rows([4, 1]), src_pool=one)
        assert torch.equal(pool, want)
        back = torch.full((n + off,), 3.0, device="cuda").to(frm)
        state_pool_copy(back[off:].view((1,) + row), _rows([5]), _rows([0]), src_pool=pool)
        assert torch.equal(back[off:].view(row), pool[5].to(frm)) and (back[:off] == 3).all()


def test_one_row_of_a_layer_and_all_rows_of_another():
    big = torch.randn((6, 3, 2, 32), device="cuda")
    ref = big.clone()
    state_pool_copy(big[:, 1], _rows([0, 0]), _rows([5, 2]), src_pool=big[4:5, 0])
    ref[[5, 2], 1] = ref[4, 0]
    assert torch.equal(big, ref)
    state_pool_copy(big[3:4, 2], _rows([5]), _rows([0]), src_pool=big[:, 1])
    ref[3, 2] = ref[5, 1]
    assert torch.equal(big, ref)
    state_pool_copy(big[:, :, :, :16], _rows([1]), _rows([0]), src_pool=big[:, :, :, 16:])
    ref[0, :, :, :16] = ref[1, :, :, 16:]
    assert torch.equal(big, ref)
    with pytest.raises(ValueError):
        state_pool_copy(big[:, 1], _rows([0]), _rows([5]), src_pool=big[4:5, 1])
