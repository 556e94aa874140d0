"""GPU tests of the state-pool row operators against list-by-list copies in
torch.  Everything but a type conversion is exact; conversions are compared
with the rounding of the fp32 value to nearest."""
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    chunk_gated_delta_rule, gated_delta_rule_decode, gated_linear_recurrence,
    gated_linear_recurrence_decode, state_pool_compact, state_pool_copy, state_pool_reset)
from tests import recurrence_testlib as R  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
ALL = [F32, BF16, F16, E4M3, E5M2]
MAX8 = {E4M3: 448.0, E5M2: 57344.0}
OUT, DUP, OVER = 16, 32, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _same(a, b):
    return torch.equal(_bits(a), _bits(b))


def _convert(v, dtype):
    if v.dtype == dtype:
        return v
    v = v.float()
    if dtype in MAX8:  # stores saturate
        v = v.clamp(-MAX8[dtype], MAX8[dtype])
    return v.to(dtype)


def _rows(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _status():
    return torch.full((1,), -1, dtype=torch.int32, device="cuda")


def _pool(seed, shape, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return _convert(torch.randn(shape, generator=gen) * scale, dtype).cuda()


SHAPES = [(1,), (3,), (5, 7), (16, 128), (2, 32, 32), (3, 5, 7), (4, 128, 128), (1, 257)]


@pytest.mark.parametrize("row", SHAPES)
@pytest.mark.parametrize("dtype", ALL)
def test_copy_inside_a_pool(row, dtype):
    pool = _pool(1, (12,) + row, dtype)
    want = pool.clone()
    src, dst = [3, 3, 3, 0, 11, 5], [1, 2, 4, 10, 9, 5]
    for s, d in zip(src, dst):
        _bits(want)  # contiguous
        want[d] = pool[s]
    st = _status()
    assert state_pool_copy(pool, _rows(src), _rows(dst), status=st) is pool
    assert st.item() == 0 and _same(pool, want)


@pytest.mark.parametrize("row", [(5, 7), (2, 32, 32), (1, 257), (16,)])
@pytest.mark.parametrize("frm", ALL)
@pytest.mark.parametrize("to", ALL)
def test_copy_converts(frm, to, row):
    src = _pool(2, (9,) + row, frm, 300.0)
    pool = _pool(3, (6,) + row, to)
    want = pool.clone()
    for s, d in ((8, 0), (2, 5), (2, 3)):
        want[d] = _convert(src[s], to)
    state_pool_copy(pool, _rows([8, 2, 2], torch.int64), _rows([0, 5, 3], torch.int64),
                    src_pool=src)
    assert _same(pool, want)


def test_copy_keeps_nan_infinity_and_saturates():
    src = torch.tensor([[float("nan"), float("inf"), -float("inf"), 1e30, -0.0, 1e-30, 3.0, 1.0]],
                       device="cuda")
    for to in ALL:
        pool = torch.zeros((1, 8), device="cuda").to(to)
        state_pool_copy(pool, _rows([0]), _rows([0]), src_pool=src)
        got = pool.float()[0]
        assert torch.isnan(got[0])
        if to in MAX8:
            assert got[1].item() == MAX8[to] and got[2].item() == -MAX8[to]
            assert got[3].item() == MAX8[to]
        else:
            assert got[1].item() == float("inf") and got[2].item() == -float("inf")
        assert got[4].item() == 0 and torch.signbit(got[4]) and got[6].item() == 3


def test_copy_lists_out_of_order():
    """Entries outside a pool are skipped, -1 is padding, the last of equal
    destinations wins, and a row that another entry overwrites is no source."""
    pool = _pool(4, (8, 16), F32)
    ref = pool.clone()
    st = _status()
    state_pool_copy(pool, _rows([0, 9, -1, 2, -7]), _rows([1, 3, 4, -1, 5]), status=st)
    want = ref.clone()
    want[1] = ref[0]
    assert st.item() == OUT and _same(pool, want)

    pool = ref.clone()
    state_pool_copy(pool, _rows([0, 1, 2, 0]), _rows([7, 7, 7, 6]), status=st)
    want = ref.clone()
    want[7], want[6] = ref[2], ref[0]
    assert st.item() == DUP and _same(pool, want)

    pool = ref.clone()
    state_pool_copy(pool, _rows([0, 1, 2, 5]), _rows([1, 2, 3, 5]), status=st)
    want = ref.clone()
    want[1] = ref[0]           # 1 -> 2 and 2 -> 3 read rows that change: skipped
    assert st.item() == OVER and _same(pool, want)

    # a swap is refused both ways
    pool = ref.clone()
    state_pool_copy(pool, _rows([0, 1]), _rows([1, 0]), status=st)
    assert st.item() == OVER and _same(pool, ref)

    # an entry outside the pool neither wins nor overwrites
    pool = ref.clone()
    state_pool_copy(pool, _rows([0, 99, 1]), _rows([7, 7, 2]), status=st)
    want = ref.clone()
    want[7], want[2] = ref[0], ref[1]
    assert st.item() == OUT and _same(pool, want)

    # between two pools nothing overlaps
    other = _pool(5, (8, 16), F32)
    pool = ref.clone()
    state_pool_copy(pool, _rows([0, 1]), _rows([1, 0]), src_pool=other, status=st)
    want = ref.clone()
    want[1], want[0] = other[0], other[1]
    assert st.item() == 0 and _same(pool, want)


@pytest.mark.parametrize("count", [0, 1, 300, 5000])
def test_copy_long_lists(count):
    """More entries than a workgroup has threads, short rows in groups."""
    rows = 6000
    src = _pool(6, (rows, 3, 4), BF16)
    pool = _pool(7, (rows, 3, 4), BF16)
    gen = torch.Generator().manual_seed(count)
    s = torch.randint(0, rows, (count,), generator=gen)
    d = torch.randint(0, rows, (count,), generator=gen)
    want = pool.clone()
    for a, b in zip(s.tolist(), d.tolist()):
        want[b] = src[a]
    st = _status()
    state_pool_copy(pool, s.cuda(), d.cuda(), src_pool=src, status=st)
    assert _same(pool, want)
    assert st.item() == (DUP if len(set(d.tolist())) < count else 0)


def test_strided_pools():
    """A layer of a [rows, layers, ...] pool, permuted states, rows that start
    off a 16-byte boundary, and copies between layers of one buffer."""
    big = _pool(8, (6, 3, 2, 32, 32), F32)
    ref = big.clone()
    state_pool_copy(big[:, 1], _rows([0]), _rows([4]))
    want = ref.clone()
    want[4, 1] = ref[0, 1]
    assert _same(big, want)
    state_pool_copy(big[:, 0], _rows([2, 4]), _rows([2, 1]), src_pool=big[:, 1])
    want[2, 0], want[1, 0] = want[2, 1], want[4, 1]
    assert _same(big, want)
    state_pool_reset(big[:, 2], _rows([0, 5]))
    want[[0, 5], 2] = 0
    assert _same(big, want)
    perm = _pool(9, (2, 7, 16, 8), BF16)
    view = perm.permute(1, 0, 3, 2)            # [7, 2, 8, 16]
    src = _pool(10, (4, 2, 8, 16), F16)
    want = view.clone()
    want[3], want[6] = src[1].to(BF16), src[0].to(BF16)
    state_pool_copy(view, _rows([1, 0]), _rows([3, 6]), src_pool=src)
    assert torch.equal(view, want)
    state_pool_reset(view, _rows([3]))
    want[3] = 0
    assert torch.equal(view, want)
    odd = torch.zeros(5 * 11 + 1, dtype=BF16, device="cuda")[1:].view(5, 11)
    odd += torch.arange(5, device="cuda", dtype=BF16)[:, None]
    state_pool_copy(odd, _rows([4]), _rows([0]))
    assert torch.equal(odd[0], odd[4]) and odd[1, 0] == 1
    # rows of one pool taken as two views
    pool = _pool(11, (10, 32), F32)
    ref = pool.clone()
    state_pool_copy(pool[5:], _rows([1]), _rows([2]), src_pool=pool[:5])
    ref[7] = ref[1]
    assert _same(pool, ref)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("row", [(1,), (5, 7), (16, 128), (4, 128, 128)])
def test_reset(dtype, row):
    pool = _pool(12, (9,) + row, dtype)
    want = pool.clone()
    for r in (0, 8, 3):
        want[r] = torch.zeros(row, device="cuda").to(dtype)
    st = _status()
    assert state_pool_reset(pool, _rows([0, 8, 3, 3, -1], torch.int64), status=st) is pool
    assert st.item() == 0 and _same(pool, want)
    state_pool_reset(pool, _rows([9, -2]), status=st)
    assert st.item() == OUT and _same(pool, want)
    state_pool_reset(pool, _rows([]), status=st)
    assert st.item() == 0 and _same(pool, want)


def _compact_ref(pool, idx):
    n = pool.shape[0]
    live = sorted({i for i in idx if 0 <= i < n})
    m = len(live)
    holes = [r for r in range(m) if r not in set(live)]
    to = dict(zip([r for r in live if r >= m], holes))
    want = pool.clone()
    for a, b in to.items():
        want[b] = pool[a]
    row_map = [-1] * n
    for r in live:
        row_map[r] = to.get(r, r)
    return want, [to.get(i, i) for i in idx], m, row_map


@pytest.mark.parametrize("rows,live,row", [
    (1, 1, (4,)), (1, 0, (4,)), (10, 4, (5, 7)), (33, 33, (8,)), (64, 1, (3, 16)),
    (65, 40, (2, 32, 32)), (1000, 500, (16,)), (5000, 3, (1,)), (40, 20, (4, 64, 64))])
@pytest.mark.parametrize("dtype,index", [(F32, torch.int32), (BF16, torch.int64),
                                         (E4M3, torch.int32)])
def test_compact(rows, live, row, dtype, index):
    gen = torch.Generator().manual_seed(rows + live)
    pool = _pool(13, (rows,) + row, dtype)
    idx = torch.randperm(rows, generator=gen)[:live].to(index)
    want, renamed, m, row_map = _compact_ref(pool, idx.tolist())
    got_map = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    st = _status()
    for _ in range(2):  # the sources stay: a repeated call does the same
        new, n = state_pool_compact(pool, idx.cuda(), row_map=got_map, status=st)
        assert n.item() == m and st.item() == 0
        assert new.dtype == index and new.tolist() == renamed
        assert got_map.tolist() == row_map
        assert _same(pool, want)


def test_compact_repeated_and_invalid_entries():
    pool = _pool(14, (12, 6), F32)
    idx = [11, 3, 11, -1, 40, 3, 9]
    want, renamed, m, _ = _compact_ref(pool, idx)
    st = _status()
    new, n = state_pool_compact(pool, _rows(idx), status=st)
    assert n.item() == m == 3 and st.item() == OUT
    assert new.tolist() == renamed and _same(pool, want)


def test_pools_without_rows_and_empty_lists():
    pool, none = torch.empty((0, 4), device="cuda"), _rows([])
    st = _status()
    assert state_pool_copy(pool, none, none) is pool
    state_pool_reset(pool, _rows([-1]), status=st)
    assert st.item() == 0
    new, n = state_pool_compact(pool, _rows([-1, 3]), status=st)
    assert n.item() == 0 and new.tolist() == [-1, 3] and st.item() == OUT
    with pytest.raises(ValueError):
        state_pool_copy(pool, _rows([0]), _rows([0]))
    full = _pool(15, (3, 4), F32)
    want = full.clone()
    state_pool_copy(full, none, none, status=st)
    assert st.item() == 0
    new, n = state_pool_compact(full, none)
    assert n.item() == 0 and new.numel() == 0 and _same(full, want)


def test_rows_of_every_alignment():
    """Rows of odd lengths at odd offsets: no access leaves its row."""
    for dtype in (F32, BF16, E4M3):
        for n in (1, 2, 3, 4, 8, 12, 15, 16, 17, 64, 100):
            for off in (0, 1, 2, 4, 8):
                base = _convert(torch.arange(5 * n + off + 3) % 7 + 1.0, dtype).cuda()
                pool = base[off:off + 5 * n].view(5, n)
                want = base.clone()
                want[off + 3 * n:off + 4 * n] = base[off + n:off + 2 * n]
                state_pool_copy(pool, _rows([1]), _rows([3]))
                want[off:off + n] = torch.zeros(n, device="cuda").to(dtype)
                state_pool_reset(pool, _rows([0]))
                assert _same(base, want), (dtype, n, off)
                wide = torch.full((4 * n + off + 2,), 9.0, device="cuda")
                want = wide.clone()
                want[off + 2 * n:off + 3 * n] = pool[3].float()
                state_pool_copy(wide[off:off + 4 * n].view(4, n), _rows([3]), _rows([2]),
                                src_pool=pool)
                assert torch.equal(wide, want), (dtype, n, off)


def test_compact_several_pools_alike():
    a, b = _pool(15, (20, 2, 32, 32), F32), _pool(16, (20, 3, 64), BF16)
    big = _pool(17, (20, 2, 8), F16)
    idx = [19, 0, 7, 15, 12]
    wants = [_compact_ref(p, idx) for p in (a, b, big[:, 1])]
    new, n = state_pool_compact([a, b, big[:, 1]], _rows(idx))
    assert n.item() == 5 and new.tolist() == wants[0][1]
    for p, w in zip((a, b, big[:, 1]), wants):
        assert torch.equal(p, w[0])


def test_compact_the_largest_pool():
    rows = 262144
    gen = torch.Generator().manual_seed(5)
    pool = torch.arange(rows, device="cuda", dtype=torch.float32).view(rows, 1).repeat(1, 4)
    idx = torch.randperm(rows, generator=gen)[: rows // 3].to(torch.int32)
    want, renamed, m, _ = None, None, rows // 3, None
    live = sorted(idx.tolist())
    alive = set(live)
    holes = [r for r in range(m) if r not in alive]
    to = dict(zip([r for r in live if r >= m], holes))
    new, n = state_pool_compact(pool, idx.cuda())
    assert n.item() == m
    assert new.tolist() == [to.get(i, i) for i in idx.tolist()]
    # row r now holds the number of the row it came from
    assert torch.equal(pool[new.long(), 0].cpu(), idx.float())


def test_graph_replay():
    pool = _pool(18, (40, 4, 32, 32), F32)
    ref = pool.clone()
    src, dst, fresh = _rows([0, 1, -1]), _rows([30, 31, -1]), _rows([5, -1])
    idx = _rows([2, 30, 31, 17])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        state_pool_copy(pool, src, dst)
        state_pool_reset(pool, fresh)
        state_pool_compact(pool, idx)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        state_pool_copy(pool, src, dst)
        state_pool_reset(pool, fresh)
        new, n = state_pool_compact(pool, idx)
    for s, d, f, live in (([0, 1, -1], [30, 31, -1], [5, -1], [2, 30, 31, 17]),
                          ([3, 3, 3], [20, 21, 22], [6, 7], [20, 21, 22, 39]),
                          ([-1, -1, -1], [-1, -1, -1], [-1, -1], [0, 1, 2, 3])):
        pool.copy_(ref)
        for t, v in ((src, s), (dst, d), (fresh, f), (idx, live)):
            t.copy_(_rows(v))
        graph.replay()
        torch.cuda.synchronize()
        eager = ref.clone()
        state_pool_copy(eager, _rows(s), _rows(d))
        state_pool_reset(eager, _rows(f))
        enew, en = state_pool_compact(eager, _rows(live))
        assert _same(pool, eager) and torch.equal(new, enew) and torch.equal(n, en)


def test_another_stream():
    pool = _pool(19, (64, 16, 64, 64), F32)
    want = pool.clone()
    want[40:48] = pool[:8]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    src, dst = _rows(list(range(8))), _rows(list(range(40, 48)))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        state_pool_copy(pool, src, dst)
    torch.cuda.current_stream().wait_stream(s)
    assert _same(pool, want)


def test_refused():
    pool = _pool(20, (8, 2, 32), F32)
    one, two = _rows([1]), _rows([1, 2])
    bad = [
        lambda: state_pool_copy(pool.cpu(), one, one),
        lambda: state_pool_copy(pool.double(), one, one),
        lambda: state_pool_copy(pool, one, two),
        lambda: state_pool_copy(pool, one, one.long()),
        lambda: state_pool_copy(pool, one.float(), one.float()),
        lambda: state_pool_copy(pool, one.cpu(), one.cpu()),
        lambda: state_pool_copy(pool, one, one, src_pool=pool[:, :1]),
        lambda: state_pool_copy(pool[:1].expand(8, 2, 32), one, one),
        lambda: state_pool_copy(pool[1:], one, one, src_pool=pool[:-1]),
        lambda: state_pool_copy(pool, one, one, src_pool=pool.view(torch.int32).view(F32)[:, :, :]
                                .transpose(1, 2).reshape(8, 2, 32)[:, :, :16]),
        lambda: state_pool_copy(pool.view(-1), one, one),
        lambda: state_pool_copy(pool, one, one, status=torch.zeros(1, device="cuda")),
        lambda: state_pool_reset(pool, one.float()),
        lambda: state_pool_reset(torch.zeros((262145, 1), device="cuda"), one),
        lambda: state_pool_compact([], one),
        lambda: state_pool_compact([pool, pool[:4].clone()], one),
        lambda: state_pool_compact(pool, two, output_indices=two),
        lambda: state_pool_compact(pool, one, output_indices=two),
        lambda: state_pool_compact(pool, one, row_map=torch.zeros(7, dtype=torch.int32,
                                                                  device="cuda")),
    ]
    ref = pool.clone()
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    assert torch.equal(pool, ref)


def test_serving_steps_together():
    """Two recurrent layers over one batch: prefill into pools, fork a
    sequence, decode, drop sequences, compact, decode on.  Every sequence
    ends with the states of its own tokens in one go."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    H, D = 2, 32
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    lens = [40, 70, 5]
    T = sum(lens)
    cu = torch.tensor([0, 40, 110, 115], dtype=torch.int32, device="cuda")
    lin = torch.full((16, H, D), 5.0, device="cuda")
    delta = torch.full((16, H, D, D), 5.0, device="cuda")
    rows = _rows([9, 4, 14])
    for pool in (lin, delta):
        state_pool_reset(pool, rows)
    x, g = rand(T, H, D), torch.rand((T, H, D), generator=gen, device="cuda")
    q, k, v = rand(T, H, D), rand(T, H, D), rand(T, H, D)
    al, be = (torch.rand((T, H), generator=gen, device="cuda") for _ in range(2))
    history = {i: [(t[a:b]) for t in (x, g, q, k, v, al, be)]
               for i, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:]))}
    gated_linear_recurrence(x, g, initial_state=lin, output_final_state=True, cu_seqlens=cu,
                            output_state=lin, state_indices=rows)
    chunk_gated_delta_rule(q, k, v, g=al, beta=be, initial_state=delta, output_final_state=True,
                           cu_seqlens=cu, output_state=delta, state_indices=rows,
                           use_qk_l2norm_in_kernel=True)

    def decode(rows, who):
        n = len(who)
        step = (rand(n, H, D), torch.rand((n, H, D), generator=gen, device="cuda"), rand(n, H, D),
                rand(n, H, D), rand(n, H, D), torch.rand((n, H), generator=gen, device="cuda"),
                torch.rand((n, H), generator=gen, device="cuda"))
        for j, w in enumerate(who):
            history[w] = [torch.cat([a, b[j:j + 1]]) for a, b in zip(history[w], step)]
        gated_linear_recurrence_decode(step[0], step[1], initial_state=lin, output_state=lin,
                                       state_indices=rows)
        gated_delta_rule_decode(step[2], step[3], step[4], g=step[5], beta=step[6],
                                initial_state=delta, output_state=delta, state_indices=rows,
                                use_qk_l2norm_in_kernel=True)

    # sequence 1 forks into 3 and 4
    for pool in (lin, delta):
        state_pool_copy(pool, _rows([4, 4]), _rows([0, 11]))
    history[3], history[4] = list(history[1]), list(history[1])
    who, rows = [0, 1, 2, 3, 4], _rows([9, 4, 14, 0, 11])
    decode(rows, who)
    decode(rows, who)
    # 0 and 4 end
    who, rows = [1, 2, 3], _rows([4, 14, 0])
    rows, n = state_pool_compact([lin, delta], rows)
    assert n.item() == 3 and sorted(rows.tolist()) == [0, 1, 2]
    decode(rows, who)
    for w, r in zip(who, rows.tolist()):
        x, g, q, k, v, al, be = history[w]
        _, _, final, ferr = R.forward(R.f64(x), R.f64(g), [x.shape[0]])
        R.check("recurrence state", lin[r:r + 1], final, ferr, F32)
        _, one = chunk_gated_delta_rule(q.contiguous(), k.contiguous(), v.contiguous(),
                                        g=al.contiguous(), beta=be.contiguous(),
                                        output_final_state=True, use_qk_l2norm_in_kernel=True)
        err = (delta[r] - one[0]).norm() / one[0].norm()
        assert err < 1e-4, err
