"""CPU tests of which two views a pool copy takes: views that share elements are
refused, interleaved ones that do not are taken, pools of one row among them."""
import ctypes
import itertools
import random

from gated_deltanet_chunked_varlen_amd import _native as nat

BASE = 0x900000
STATE = nat.ERR_CODE["GDN_ERR_STATE"]


class View:
    """A view of a float32 buffer of `shape`: start element, shape, strides."""

    def __init__(self, shape, start=0, strides=None):
        self.shape, self.start = tuple(shape), start
        if strides is None:
            strides, step = [], 1
            for n in reversed(shape):
                strides.insert(0, step)
                step *= n
        self.strides = tuple(strides)

    def __getitem__(self, key):
        key = key if isinstance(key, tuple) else (key,)
        start, shape, strides = self.start, [], []
        for i, (n, st) in enumerate(zip(self.shape, self.strides)):
            k = key[i] if i < len(key) else slice(None)
            if isinstance(k, int):
                start += k * st
                continue
            a, b, c = k.indices(n)
            start += a * st
            shape.append(len(range(a, b, c)))
            strides.append(st * c)
        return View(shape, start, strides)

    def elements(self):
        return {self.start + sum(i * s for i, s in zip(at, self.strides))
                for at in itertools.product(*map(range, self.shape))}


def _check(dst, src):
    p = nat.PoolParams()
    pad = 4 - len(dst.shape)
    for name, v in (("dst", dst), ("src", src)):
        # as the binding passes them: 1 for a dimension that is never stepped over
        st = [v.strides[0] if v.shape[0] > 1 else 1] + [1] * pad
        st += [s if n > 1 else 1 for n, s in zip(v.shape[1:], v.strides[1:])]
        setattr(p, name, ctypes.c_void_p(BASE + 4 * v.start))
        setattr(p, name + "_strides", nat._i64x4(*st))
        setattr(p, name + "_pool_rows", v.shape[0])
    p.extent = nat._i64x3(*([1] * pad + list(dst.shape[1:])))
    p.src_rows = p.dst_rows = ctypes.c_void_p(0x1000)
    p.count = 2
    return nat.lib().gdn_validate_pool_host(ctypes.byref(p), 0)


def test_pools_of_one_row():
    big = View((6, 3, 2, 8))
    assert _check(big[:, 0], big[:, 1]) == 0
    for r in (0, 2, 5):
        assert _check(big[r:r + 1, 0], big[:, 1]) == 0
        assert _check(big[:, 0], big[r:r + 1, 1]) == 0
        assert _check(big[r:r + 1, 2], big[:, 1]) == 0
        # a row of the other view itself
        assert _check(big[r:r + 1, 1], big[:, 1]) == STATE
        assert _check(big[:, 1], big[r:r + 1, 1]) == STATE
    assert _check(big[1:2, 1], big[1:2, 1]) == 0  # one view
    assert _check(big[1:2, 1], big[1:2, 0]) == 0
    assert _check(big[0:1, 0:2], big[0:1, 1:3]) == STATE


def test_views_interleaved_inside_the_rows():
    big = View((5, 4, 16))
    assert _check(big[:, :2], big[:, 2:]) == 0
    assert _check(big[:, :, :8], big[:, :, 8:]) == 0
    assert _check(big[:, :, 0::2], big[:, :, 1::2]) == 0
    assert _check(big[1:, :, :8], big[:-1, :, 8:]) == 0
    assert _check(big[:, :, :9], big[:, :, 7:]) == STATE
    assert _check(big[:, 0:3], big[:, 1:4]) == STATE
    assert _check(big[1:], big[:-1]) == STATE
    assert _check(big[0::2], big[1::2]) == 0


def test_random_pairs_of_views():
    """Against the elements themselves: what shares some is always refused; what
    shares none is taken where the strides are equal."""
    rng = random.Random(0)
    taken = refused = 0
    for _ in range(8000):
        shape = tuple(rng.randint(1, 5) for _ in range(4))
        big = View(shape)

        def cut():
            key = []
            for n in shape:
                a = rng.randint(0, n - 1)
                key.append(slice(a, rng.randint(a + 1, n), rng.choice([1, 1, 2])))
            return big[tuple(key)]

        dst, src = cut(), cut()
        if dst.shape[1:] != src.shape[1:]:
            continue
        if (dst.start, dst.strides) == (src.start, src.strides):
            continue  # the same view (of some of the rows)
        rc = _check(dst, src)
        shared = bool(dst.elements() & src.elements())
        assert rc in (0, STATE)
        if shared:
            # one view, where only steps that are never taken differ
            same = dst.start == src.start and all(
                a == b or n <= 1 or m <= 1 for a, b, n, m in
                zip(dst.strides, src.strides, dst.shape, src.shape))
            assert rc == STATE or same
        elif all(a == b or n <= 1 or m <= 1 for a, b, n, m in
                 zip(dst.strides, src.strides, dst.shape, src.shape)):
            assert rc == 0, (shape, dst.__dict__, src.__dict__)
        taken += rc == 0
        refused += rc == STATE
    assert taken > 100 and refused > 100
