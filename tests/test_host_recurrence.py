"""CPU tests of the recurrence's and the pool operators' host side: struct
layouts, argument checks and their codes, workspace sizes.  No compute call is
made."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from gated_deltanet_chunked_varlen_amd import _native as nat
from tests.conftest import ROOT

FAKE = ctypes.c_void_p(0x1000)


def code(name):
    return nat.ERR_CODE[name]


@pytest.mark.parametrize("struct,cls", [("gdn_recurrence_params", nat.RecurrenceParams),
                                        ("gdn_pool_params", nat.PoolParams)])
def test_struct_layout_matches_the_header(struct, cls):
    fields = [f for f, _ in cls._fields_]
    src = ['#include <stdio.h>', '#include <stddef.h>',
           '#include "%s"' % os.path.join(ROOT, "include", "gdn_prefill.h"),
           "int main(void) {", '  printf("%%zu\\n", sizeof(%s));' % struct]
    src += ['  printf("%%zu\\n", offsetof(%s, %s));' % (struct, f) for f in fields]
    src += ["  return 0;", "}"]
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(c, "w").write("\n".join(src))
        subprocess.check_call(["gcc", "-std=c99", c, "-o", exe])
        got = [int(x) for x in subprocess.check_output([exe]).split()]
    assert got[0] == ctypes.sizeof(cls)
    assert got[1:] == [getattr(cls, f).offset for f in fields]


def test_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "gdn_prefill.h")).read()
    for name, value in (("GDN_RECURRENCE_CHUNK", nat.RECURRENCE_CHUNK),
                        ("GDN_POOL_MAX_ROWS", nat.POOL_MAX_ROWS),
                        ("GDN_STATUS_POOL_ROW", nat.STATUS_POOL_ROW),
                        ("GDN_STATUS_POOL_DUPLICATE", nat.STATUS_POOL_DUPLICATE),
                        ("GDN_STATUS_POOL_OVERLAP", nat.STATUS_POOL_OVERLAP)):
        line = [l for l in src.splitlines() if l.startswith("#define %s " % name)][0]
        assert int(line.split()[2].rstrip("u")) == value
    for bit in (16, 32, 64):
        assert nat.status_string(bit) != "unknown code"


def _rec(mode=0, **kw):
    p = nat.RecurrenceParams()
    p.total_tokens, p.num_seqs, p.num_heads, p.head_size = 1000, 3, 4, 32
    p.x_dtype, p.g_dtype = nat.GDN_BF16, nat.GDN_F32
    p.x = p.g = p.output = p.doutput = p.dx = p.dg = FAKE
    p.cu_seqlens = FAKE
    if mode == 2:
        p.total_tokens, p.cu_seqlens = 3, None
    for f, v in kw.items():
        setattr(p, f, v)
    return p


def _check(p, mode=0, workspace=True):
    L = nat.lib()
    if workspace:
        p.workspace = ctypes.c_void_p(0x10000)
        p.workspace_bytes = L.gdn_recurrence_workspace_size(ctypes.byref(p), int(mode == 1))
    return L.gdn_validate_recurrence_host(ctypes.byref(p), mode)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_recurrence_accepted(mode):
    for kw in (dict(), dict(x_dtype=nat.GDN_F32), dict(g_dtype=nat.GDN_BF16),
               dict(head_size=5), dict(g_per_head=1), dict(g_per_head=1, head_size=128),
               dict(x_stride=128), dict(x_stride=1000, g_stride=129),
               dict(initial_state=FAKE, initial_state_dtype=nat.GDN_FP8_E4M3),
               dict(x=ctypes.c_void_p(0x1002))):
        assert _check(_rec(mode, **kw), mode) == 0, kw


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("kw,err", [
    (dict(num_heads=0), "GDN_ERR_SHAPE"),
    (dict(head_size=0), "GDN_ERR_SHAPE"),
    (dict(head_size=-3), "GDN_ERR_SHAPE"),
    (dict(total_tokens=-1), "GDN_ERR_SHAPE"),
    (dict(num_seqs=-1), "GDN_ERR_SHAPE"),
    (dict(total_tokens=2 ** 31), "GDN_ERR_SHAPE"),
    (dict(num_heads=2 ** 20, head_size=2 ** 12), "GDN_ERR_SHAPE"),
    (dict(g_per_head=2), "GDN_ERR_SHAPE"),
    (dict(g_per_head=1, head_size=48), "GDN_ERR_SHAPE"),
    (dict(x_dtype=nat.GDN_FP8_E4M3), "GDN_ERR_DTYPE"),
    (dict(g_dtype=nat.GDN_F16), "GDN_ERR_DTYPE"),
    (dict(x=None), "GDN_ERR_NULL"),
    (dict(g=None), "GDN_ERR_NULL"),
    (dict(x_stride=127), "GDN_ERR_STRIDES"),
    (dict(g_stride=-128), "GDN_ERR_STRIDES"),
    (dict(x=ctypes.c_void_p(0x1001)), "GDN_ERR_ALIGN"),
    (dict(g=ctypes.c_void_p(0x1002)), "GDN_ERR_ALIGN"),
    (dict(initial_state=FAKE, initial_state_dtype=9), "GDN_ERR_DTYPE"),
    (dict(initial_state=FAKE, initial_state_stride=5), "GDN_ERR_STRIDES"),
    (dict(initial_state=ctypes.c_void_p(0x1001)), "GDN_ERR_ALIGN"),
])
def test_recurrence_refused(mode, kw, err):
    assert _check(_rec(mode, **kw), mode) == code(err)


@pytest.mark.parametrize("mode,kw,err", [
    (0, dict(cu_seqlens=None), "GDN_ERR_SHAPE"),
    (0, dict(cu_seqlens_type=4), "GDN_ERR_DTYPE"),
    (0, dict(output=None), "GDN_ERR_NULL"),
    (0, dict(output=ctypes.c_void_p(0x1001)), "GDN_ERR_ALIGN"),
    (0, dict(output_final_state=1), "GDN_ERR_STATE"),
    (0, dict(output_final_state=1, output_state=FAKE, output_state_dtype=7), "GDN_ERR_DTYPE"),
    (0, dict(output_final_state=1, output_state=FAKE, output_state_stride=1), "GDN_ERR_STRIDES"),
    (0, dict(state_indices=FAKE), "GDN_ERR_STATE"),
    (0, dict(state_indices=FAKE, pool_size=4, state_indices_type=3), "GDN_ERR_DTYPE"),
    (0, dict(chunk_states=ctypes.c_void_p(0x1002)), "GDN_ERR_ALIGN"),
    (1, dict(state_indices=FAKE, pool_size=4), "GDN_ERR_STATE"),
    (1, dict(doutput=None), "GDN_ERR_NULL"),
    (1, dict(dx=None), "GDN_ERR_NULL"),
    (1, dict(dg=None), "GDN_ERR_NULL"),
    (1, dict(doutput_stride=64), "GDN_ERR_STRIDES"),
    (1, dict(dinitial_state=ctypes.c_void_p(0x1002)), "GDN_ERR_ALIGN"),
    (2, dict(total_tokens=4), "GDN_ERR_SHAPE"),
    (2, dict(cu_seqlens=FAKE), "GDN_ERR_SHAPE"),
    (2, dict(chunk_states=FAKE), "GDN_ERR_STATE"),
])
def test_recurrence_refused_by_mode(mode, kw, err):
    assert _check(_rec(mode, **kw), mode) == code(err)


def test_recurrence_null_and_mode():
    L = nat.lib()
    assert L.gdn_validate_recurrence_host(None, 0) == code("GDN_ERR_NULL")
    assert L.gdn_validate_recurrence_host(ctypes.byref(_rec()), 3) == code("GDN_ERR_SHAPE")
    assert L.gdn_recurrence_workspace_size(None, 0) == 0
    assert L.gdn_recurrence(None, None) == code("GDN_ERR_NULL")
    assert L.gdn_recurrence_backward(None, None) == code("GDN_ERR_NULL")
    assert L.gdn_recurrence_decode(None, None) == code("GDN_ERR_NULL")


def test_recurrence_workspace():
    L = nat.lib()
    size = lambda back=0, **kw: L.gdn_recurrence_workspace_size(  # noqa: E731
        ctypes.byref(_rec(**kw)), back)
    # one tile and few sequences need none
    assert size(total_tokens=64) == 0 and size(back=1, total_tokens=64) == 0
    assert size(total_tokens=64, num_seqs=64) > 0
    # the backward pass keeps the states itself where the caller did not
    assert size(back=1) >= size() + 16 * 128 * 4
    assert size(back=1, chunk_states=FAKE) == size()
    p = _rec()
    assert _check(p, workspace=False) == code("GDN_ERR_WORKSPACE")
    need = size()
    p.workspace, p.workspace_bytes = ctypes.c_void_p(0x10000), need - 1
    assert _check(p, workspace=False) == code("GDN_ERR_WORKSPACE")
    p.workspace, p.workspace_bytes = ctypes.c_void_p(0x10010), need
    assert _check(p, workspace=False) == code("GDN_ERR_ALIGN")


def _pool(**kw):
    p = nat.PoolParams()
    p.extent = nat._i64x3(4, 8, 16)
    p.src, p.dst = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x900000)
    p.src_pool_rows, p.dst_pool_rows = 10, 20
    p.src_rows = p.dst_rows = FAKE
    p.count = 5
    for f, v in kw.items():
        setattr(p, f, v)
    return p


def _pool_check(p, mode):
    return nat.lib().gdn_validate_pool_host(ctypes.byref(p), mode)


def test_pool_accepted():
    S = nat._i64x4
    for mode in (0, 1, 2):
        assert _pool_check(_pool(), mode) == 0
        assert _pool_check(_pool(count=0, src_rows=None, dst_rows=None), mode) == 0
        assert _pool_check(_pool(dst_strides=S(600, 128, 1, 8)), mode) == 0
    # one view, and interleaved rows of one buffer
    assert _pool_check(_pool(src=0x900000, src_pool_rows=20), 0) == 0
    two = S(1024, 128, 16, 1)
    assert _pool_check(_pool(src=0x900000 + 512 * 4, src_strides=two, dst_strides=two,
                             src_pool_rows=20), 0) == 0


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("kw,err", [
    (dict(extent=nat._i64x3(4, 0, 16)), "GDN_ERR_SHAPE"),
    (dict(extent=nat._i64x3(2 ** 31 - 1, 2 ** 31 - 1, 16)), "GDN_ERR_SHAPE"),
    (dict(dst_pool_rows=-1), "GDN_ERR_SHAPE"),
    (dict(dst_pool_rows=262145), "GDN_ERR_SHAPE"),
    (dict(count=-1), "GDN_ERR_SHAPE"),
    (dict(dst_dtype=5), "GDN_ERR_DTYPE"),
    (dict(rows_type=2), "GDN_ERR_DTYPE"),
    (dict(dst=None), "GDN_ERR_NULL"),
    (dict(dst_rows=None), "GDN_ERR_NULL"),
    (dict(dst=0x900002), "GDN_ERR_ALIGN"),
    (dict(dst_strides=nat._i64x4(512, 128, 16, -1)), "GDN_ERR_STRIDES"),
    (dict(dst_strides=nat._i64x4(511, 128, 16, 1)), "GDN_ERR_STRIDES"),
])
def test_pool_refused(mode, kw, err):
    assert _pool_check(_pool(**kw), mode) == code(err)


@pytest.mark.parametrize("kw,err", [
    (dict(src=None), "GDN_ERR_NULL"),
    (dict(src_rows=None), "GDN_ERR_NULL"),
    (dict(src_dtype=-1), "GDN_ERR_DTYPE"),
    (dict(src_pool_rows=262145), "GDN_ERR_SHAPE"),
    (dict(src=0x100001, src_dtype=1), "GDN_ERR_ALIGN"),
    (dict(src_strides=nat._i64x4(512, 100, 16, 1)), "GDN_ERR_STRIDES"),
    # views that share rows: shifted by one row, by part of a row, another type
    (dict(src=0x900000 + 512 * 4), "GDN_ERR_STATE"),
    (dict(src=0x900000 + 64), "GDN_ERR_STATE"),
    (dict(src=0x900000, src_dtype=1), "GDN_ERR_STATE"),
    (dict(src=0x900000 + 256 * 4, src_strides=nat._i64x4(1024, 128, 16, 1),
          dst_strides=nat._i64x4(1024, 128, 16, 1)), "GDN_ERR_STATE"),
])
def test_pool_copy_refused(kw, err):
    assert _pool_check(_pool(**kw), 0) == code(err)


def test_pool_null():
    L = nat.lib()
    assert L.gdn_validate_pool_host(None, 0) == code("GDN_ERR_NULL")
    assert L.gdn_validate_pool_host(ctypes.byref(_pool()), 3) == code("GDN_ERR_SHAPE")
    assert L.gdn_pool_copy(None, None) == code("GDN_ERR_NULL")
    assert L.gdn_pool_reset(None, None) == code("GDN_ERR_NULL")
    assert L.gdn_pool_compact(None, None, None, None, None) == code("GDN_ERR_NULL")


def test_python_calls_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import gated_deltanet_chunked_varlen_amd as gdn
    x, i = torch.zeros((4, 2, 32)), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gated_linear_recurrence(x, x)
    with pytest.raises(ValueError):
        gdn.gated_linear_recurrence_backward(x, x, x)
    with pytest.raises(ValueError):
        gdn.gated_linear_recurrence_decode(x, x)
    for call in (lambda: gdn.state_pool_copy(x, i, i), lambda: gdn.state_pool_reset(x, i),
                 lambda: gdn.state_pool_compact(x, i), lambda: gdn.state_pool_reset(3, i)):
        with pytest.raises(ValueError):
            call()
