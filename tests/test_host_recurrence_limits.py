"""CPU tests of the largest calls the recurrence and the pool operators take: what
the host accepts, a grid holds and a kernel's loops count."""
import ctypes

import pytest

from gated_deltanet_chunked_varlen_amd import _native as nat

FAKE = ctypes.c_void_p(0x1000)
SHAPE = nat.ERR_CODE["GDN_ERR_SHAPE"]


def _rec(mode, T, N, H, D):
    p = nat.RecurrenceParams()
    p.total_tokens, p.num_seqs, p.num_heads, p.head_size = T, N, H, D
    p.x_dtype, p.g_dtype = nat.GDN_BF16, nat.GDN_F32
    p.x = p.g = p.output = p.doutput = p.dx = p.dg = FAKE
    p.cu_seqlens = FAKE if mode != 2 else None
    L = nat.lib()
    p.workspace = ctypes.c_void_p(0x10000)
    p.workspace_bytes = L.gdn_recurrence_workspace_size(ctypes.byref(p), int(mode == 1))
    return L.gdn_validate_recurrence_host(ctypes.byref(p), mode)


def test_decode_calls_that_fit_a_grid():
    # one thread per four channels, workgroups of 256 in fewer than 2^32 threads
    assert _rec(2, 2 ** 21, 2 ** 21, 1, 8188) == 0
    assert _rec(2, 2 ** 21, 2 ** 21, 1, 8192) == SHAPE
    assert _rec(2, 2 ** 21, 2 ** 21, 4, 4096) == SHAPE
    assert _rec(2, 2 ** 30 - 64, 2 ** 30 - 64, 1, 16) == 0
    assert _rec(2, 2 ** 30 - 63, 2 ** 30 - 63, 1, 16) == SHAPE


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_sequences_that_32_bits_count(mode):
    T = lambda n: n if mode == 2 else 10  # noqa: E731
    assert _rec(mode, T(2 ** 30), 2 ** 30, 1, 1) == 0
    assert _rec(mode, T(2 ** 30 + 1), 2 ** 30 + 1, 1, 1) == SHAPE
    assert _rec(mode, T(2 ** 31 - 65), 2 ** 31 - 65, 1, 1) == SHAPE


def test_empty_sequences_fit_the_grid_of_a_scan():
    empties = nat.lib()._ZN3gdn11rec_emptiesEjii
    empties.restype = ctypes.c_int32
    empties.argtypes = [ctypes.c_uint32, ctypes.c_int32, ctypes.c_int32]
    most = 2 ** 22 - 1
    for ncb in (1, 2, 3, 16, 65535, 65536, 102300, 1048575, 1398101, 2 ** 20 + 1, 2 ** 21):
        for tiles in {1, 2, most // ncb}:
            units = tiles * ncb
            if units > most:
                continue
            for n in (0, 1, 64, 65, 4096, 2 ** 30):
                e = empties(units, ncb, n)
                assert (e > 0) == (n > 0) and e <= 64 and 64 * (e - 1) <= n
                assert (units + e * ncb) * 512 < 2 ** 32
    assert empties(16, 16, 100) == 2 and empties(16, 16, 10 ** 6) == 64


def test_lists_of_a_copy():
    """A copy compares its entries with each other: as many as a pool has rows."""
    p = nat.PoolParams()
    p.extent = nat._i64x3(1, 1, 4)
    p.src, p.dst = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x900000)
    p.src_pool_rows = p.dst_pool_rows = 16
    p.src_rows = p.dst_rows = FAKE
    check = lambda mode: nat.lib().gdn_validate_pool_host(ctypes.byref(p), mode)  # noqa: E731
    for mode in (0, 1, 2):
        p.count = nat.POOL_MAX_ROWS
        assert check(mode) == 0
        p.count += 1
        assert check(mode) == (SHAPE if mode == 0 else 0)
