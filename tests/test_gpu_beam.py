"""GPU tests of beam search over state pools: selection against a full sort in
fp64, rows of pools against the definition."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import (  # noqa: E402
    _native as nat, beam_select, state_pool_reorder)

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _select(logits, scores, m):
    """(scores, parents, tokens) by a full sort of every continuation."""
    x = logits.float().cpu().numpy().astype(np.float64)
    s = scores.cpu().numpy().astype(np.float64)
    x = np.where(np.isnan(x), -INF, x)
    B, K, V = x.shape
    val = np.full((B, K, V), -INF)
    for b in range(B):
        for k in range(K):
            top = x[b, k].max()
            if not s[b, k] > -INF or top == -INF:
                continue
            away = np.where(x[b, k] == top, 0.0, x[b, k] - (0.0 if np.isinf(top) else top))
            if np.isinf(top):
                away = np.where(x[b, k] == top, 0.0, -INF)
            val[b, k] = s[b, k] + (away - np.log(np.exp(away).sum()))
    flat = val.reshape(B, -1)
    at = np.stack([np.lexsort((np.arange(K * V), -flat[b]))[:m] for b in range(B)])
    return np.take_along_axis(flat, at, 1), at // V, at % V


def _check(logits, scores, m, **kw):
    got = beam_select(logits, scores, m, **kw)
    want = _select(logits, scores, m)
    assert [t.dtype for t in got] == [F32, torch.int32, torch.int32]
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[2].cpu().numpy(), want[2])
    g, w = got[0].cpu().numpy().astype(np.float64), want[0]
    fin = np.isfinite(w)
    assert np.array_equal(g[~fin], w[~fin])
    # fp32 sums of positive terms, each off by its argument's rounding (at most
    # 2^-24 |logit - largest| e^-..., below 2^-24), its step 2^-23 and 35 sums;
    # log halves none of it; then the result's own rounding
    assert (np.abs(g[fin] - w[fin]) <= 2.0 ** -24 * (40 + np.abs(w[fin]))).all()


def _make(seed, B, K, V, dtype, by=3.0):
    gen = torch.Generator().manual_seed(seed)
    return ((by * torch.randn((B, K, V), generator=gen)).to(dtype).cuda(),
            (-10 * torch.rand((B, K), generator=gen)).cuda())


@pytest.mark.parametrize("B,K,V,m,dtype", [
    (1, 1, 1, 1, F32), (1, 1, 7, 7, F32), (3, 2, 5, 10, BF16), (2, 4, 1000, 8, F16),
    (1, 4, 32001, 8, F32), (2, 64, 301, 64, F32), (1, 3, 2049, 17, F32), (5, 8, 8193, 16, BF16),
    (40, 16, 2000, 32, F16), (1, 64, 70000, 64, F32), (130, 4, 16400, 4, BF16), (1, 2, 200001, 2, F32),
])
def test_select(B, K, V, m, dtype):
    _check(*_make(B + K + V, B, K, V, dtype), m)


def test_default_is_as_many_as_beams():
    logits, scores = _make(1, 2, 5, 300, F32)
    assert beam_select(logits, scores)[0].shape == (2, 5)


@pytest.mark.parametrize("V,m", [(9000, 64), (300, 16), (20000, 16)])
def test_ties(V, m):
    """Logits of few values, rows all alike, beams alike: the lowest beam and token."""
    gen = torch.Generator().manual_seed(V)
    logits = torch.randint(-2, 2, (4, 4, V), generator=gen).float().cuda()
    logits[1] = 1.5
    logits[2, 3] = logits[2, 0]
    logits[3] = logits[3, :1]
    scores = -torch.arange(4.0).repeat(4, 1).cuda()
    scores[2, 3] = scores[2, 0]
    scores[3] = -0.25
    _check(logits, scores, m)
    _check(logits * 0.0 * -1.0, scores, m)  # zeros of both signs
    _check(torch.where(logits > 0, 0.0, -0.0), scores, m)


def test_ordered_logits():
    """All of the largest ones in one thread's or one part's share."""
    for V in (8192, 30000):
        up = torch.arange(V, dtype=F32, device="cuda").repeat(1, 2, 1) * 1e-3
        scores = torch.zeros((1, 2), device="cuda")
        _check(up, scores - torch.tensor([[0.0, 1e-4]], device="cuda"), 64)
        _check(up.flip(-1).contiguous(), scores - torch.tensor([[0.0, 1e-4]], device="cuda"), 64)


def test_nothing_to_choose():
    """Ended beams, rows that a mask leaves nothing of, NaN and infinite logits."""
    logits, scores = _make(7, 8, 3, 2500, F32)
    scores[0] = -INF                      # every beam has ended
    scores[1, 1] = -INF
    scores[2, 0] = float("nan")
    logits[3] = -INF                      # nothing is left
    logits[4, 1] = -INF
    logits[5, :, 3:] = -INF               # fewer than there are places
    logits[6, 0, 5] = float("nan")
    logits[7, 1, 9] = INF
    logits[7, 1, 700] = INF
    for m in (3, 16, 40):
        _check(logits, scores, m)
    _check(torch.full_like(logits, float("nan")), scores, 5)
    low = torch.full((2, 2, 300), torch.finfo(F32).min, device="cuda")
    low[0, 0, 7] = 0.0
    _check(low, scores[:2, :2].contiguous().fill_(-1.0), 9)


def test_large_logits_and_scores():
    logits, scores = _make(8, 2, 4, 5000, F32, by=1e4)
    got = beam_select(logits, scores - 1e6, 8)
    want = _select(logits, scores - 1e6, 8)
    assert np.array_equal(got[2].cpu().numpy()[:, 0], want[2][:, 0])
    assert np.allclose(got[0].cpu().numpy(), want[0], rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("V", [50, 3000, 20001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scores_that_are_equal_for_unequal_logits(V, dtype):
    """Scores that 64 bits do not tell apart, or infinite ones, are ties: the lowest
    token, whatever its logit."""
    logits, scores = _make(V, 7, 3, V, dtype)
    scores[0] = torch.finfo(F32).min                  # beams as good as dead
    scores[1, 1:] = torch.finfo(F32).min
    logits[1, 0, 2:] = -INF                           # two tokens are allowed
    scores[2] = torch.tensor([-1e30, INF, -1e30])
    logits[3, 1, V // 2] = INF                        # the others have no share
    logits[3, 1, V - 1] = INF
    scores[3, 0] = -INF
    scores[3, 2] = float("nan")
    logits[4, :, V - 3] = 1e30
    logits[5, :, ::2] = -INF
    scores[5] = -1e30
    logits[6, 0] = INF
    logits[6, 1, 7] = INF
    scores[6, 2] = -INF
    for m in (1, 5, 16, 40):
        _check(logits, scores, m)
        _check(logits[:, 1:2].contiguous(), scores[:, 1:2].contiguous(), m)


def test_strides_and_odd_addresses():
    logits, scores = _make(9, 3, 4, 1001, BF16)
    wide = torch.zeros((3, 4, 1100), dtype=BF16, device="cuda")
    for off in (0, 8, 13):
        view = wide[:, :, off:off + 1001]
        view.copy_(logits)
        _check(view, scores, 8)
    _check(torch.zeros((5, 1, 30), device="cuda")[::2], torch.zeros((3, 1), device="cuda"), 4)


def test_select_refusals():
    logits, scores = _make(10, 2, 4, 100, F32)
    for call in (
            lambda: beam_select(logits, scores, 0), lambda: beam_select(logits, scores, 65),
            lambda: beam_select(logits[:, :, :3].contiguous(), scores, 13),
            lambda: beam_select(logits.to(torch.float64), scores), lambda: beam_select(logits[0], scores),
            lambda: beam_select(logits, scores[:1]), lambda: beam_select(logits, scores.to(BF16)),
            lambda: beam_select(logits.transpose(0, 1), scores.t().contiguous()),
            lambda: beam_select(logits[:, :, ::2], scores), lambda: beam_select(logits, scores.cpu()),
            lambda: beam_select(logits.clone().requires_grad_(), scores),
            lambda: beam_select(torch.zeros((1, 65, 4), device="cuda"), torch.zeros((1, 65), device="cuda")),
            lambda: beam_select(logits.expand(2, 4, 100)[:, :1].expand(2, 4, 100), scores)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        beam_select(logits, scores, "8")
    assert beam_select(logits[:0], scores[:0], 4)[1].shape == (0, 4)


# -------------------------------------------------------------------- reorder

def _reorder(pool, idx, parents):
    """(pool, indices) by the definition; rows outside the pool are handed on."""
    new, rows = [], pool.shape[0]
    out = pool.clone()
    for b, p in enumerate(parents):
        K = len(p)
        own = idx[b * K:(b + 1) * K]
        kept, left = set(), [k for k in range(K) if k not in p]
        for q in p:
            if 0 <= q < K and q not in kept:
                kept.add(q)
                new.append(own[q])
                continue
            to = own[left.pop(0)]
            new.append(to)
            if 0 <= q < K and 0 <= to < rows and 0 <= own[q] < rows:
                out[to] = pool[own[q]]
    return out, new


def _bytes(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("B,K,shape,dtype,itype", [
    (1, 1, (4,), F32, torch.int32), (2, 4, (16, 128), F32, torch.int32), (3, 5, (3, 7), BF16, torch.int64),
    (2, 64, (5,), torch.float8_e4m3fn, torch.int32), (4, 3, (2, 64, 65), F16, torch.int32),
    (1, 8, (16, 128, 128), F32, torch.int64), (50, 7, (33,), F32, torch.int32)])
def test_reorder(B, K, shape, dtype, itype):
    gen = torch.Generator().manual_seed(B * K)
    rows = B * K + 5
    pool = torch.randn((rows,) + shape, generator=gen).to(dtype).cuda()
    idx = torch.randperm(rows, generator=gen)[:B * K].to(itype).cuda()
    for kind in range(4):
        if kind == 0:
            parents = torch.randint(K, (B, K), generator=gen)
        elif kind == 1:
            parents = torch.arange(K).repeat(B, 1)
        elif kind == 2:
            parents = torch.full((B, K), K - 1)
        else:
            parents = torch.stack([torch.randperm(K, generator=gen) for _ in range(B)])
        want, new = _reorder(pool, idx.tolist(), parents.tolist())
        status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
        got = pool.clone()
        res = state_pool_reorder(got, idx, parents.to(itype).cuda(), status=status)
        assert res.dtype == itype and res.tolist() == new and status.item() == 0
        assert torch.equal(_bytes(got), _bytes(want))


def test_reorder_of_many_pools_and_views():
    """A model's layers: more pools than one launch takes, of several types and
    shapes, slices of a wider tensor among them."""
    gen = torch.Generator().manual_seed(3)
    rows, B, K = 20, 2, 4
    deep = torch.randn((rows, 9, 4, 33), generator=gen).cuda()
    pools = [deep[:, i] for i in range(9)]
    pools += [torch.randn((rows, 3, 40), generator=gen).to(t).cuda() for t in (F32, BF16, F16)] * 3
    pools.append(torch.randn((4, rows, 6), generator=gen).cuda().transpose(0, 1))
    pools = [p if i < 9 else p.clone() if p.is_contiguous() else p for i, p in enumerate(pools)]
    idx = torch.randperm(rows, generator=gen)[:B * K].to(torch.int32).cuda()
    parents = torch.tensor([[2, 2, 0, 2], [1, 1, 1, 1]], dtype=torch.int32)
    want = [_reorder(p.clone(), idx.tolist(), parents.tolist()) for p in pools]
    out = torch.empty_like(idx)
    res = state_pool_reorder(pools, idx, parents.cuda(), output_indices=out)
    assert res is out and res.tolist() == want[0][1]
    for p, (w, _) in zip(pools, want):
        assert torch.equal(_bytes(p), _bytes(w))


def test_reorder_of_bad_entries():
    pool = torch.randn((6, 8), device="cuda")
    cases = [  # indices, parents, status
        ([0, 1, 2, 3], [[3, -1, 3, 7]], nat.STATUS_POOL_ROW),
        ([0, -1, 2, 3], [[1, 1, 0, 0]], 0),
        ([0, 9, 2, 3], [[1, 1, 0, 0]], nat.STATUS_POOL_ROW),
        ([0, -1, -1, 3], [[0, 0, 0, -1]], 0),
        ([0, 1, 1, 3], [[0, 1, 2, 3]], nat.STATUS_POOL_DUPLICATE),
    ]
    for idx, parents, bits in cases:
        want, new = _reorder(pool, idx, parents)
        got, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        res = state_pool_reorder(got, torch.tensor(idx, device="cuda"),
                                 torch.tensor(parents, device="cuda"), status=status)
        assert res.tolist() == new and status.item() == bits, idx
        assert torch.equal(got, want)


def test_reorder_refusals():
    pool = torch.randn((6, 8), device="cuda")
    idx, par = torch.arange(4, device="cuda"), torch.zeros((1, 4), dtype=torch.int64, device="cuda")
    for call in (
            lambda: state_pool_reorder([], idx, par), lambda: state_pool_reorder(pool, idx, par.int()),
            lambda: state_pool_reorder(pool, idx[:3], par), lambda: state_pool_reorder(pool, idx, par[0]),
            lambda: state_pool_reorder([pool, pool[:5]], idx, par),
            lambda: state_pool_reorder(pool, idx, par, output_indices=idx),
            lambda: state_pool_reorder(pool, idx, par, output_indices=par[0]),
            lambda: state_pool_reorder(pool[:, :1].expand(6, 8), idx, par),
            lambda: state_pool_reorder(pool.clone().requires_grad_(), idx, par),
            lambda: state_pool_reorder(pool.cpu(), idx, par),
            lambda: state_pool_reorder(pool, torch.zeros(65, dtype=torch.int64, device="cuda"),
                                       torch.zeros((1, 65), dtype=torch.int64, device="cuda"))):
        before = pool.clone()
        with pytest.raises(ValueError):
            call()
        assert torch.equal(pool, before)
