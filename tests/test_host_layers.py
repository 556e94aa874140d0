"""CPU tests of the host side of the short convolution, the selective scan and beam
search: struct layouts, argument checks and their codes, workspace sizes.  No
compute call is made."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from gated_deltanet_chunked_varlen_amd import _native as nat
from tests.conftest import ROOT

FAKE = ctypes.c_void_p(0x1000)


def far(k):
    return ctypes.c_void_p(0x1000 + (k << 32))


def code(name):
    return nat.ERR_CODE[name]


@pytest.mark.parametrize("struct,cls", [
    ("gdn_convolution_params", nat.ConvolutionParams), ("gdn_scan_params", nat.ScanParams),
    ("gdn_beam_params", nat.BeamParams), ("gdn_reorder_pool", nat.ReorderPool),
    ("gdn_reorder_params", nat.ReorderParams)])
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
    line = [l for l in src.splitlines() if l.startswith("#define GDN_BEAM_MAX ")][0]
    assert int(line.split()[2]) == nat.BEAM_MAX


# ---------------------------------------------------------------- convolution

def _conv(mode=0, **kw):
    p = nat.ConvolutionParams()
    p.total_tokens, p.num_seqs, p.channels, p.width = 1000, 3, 96, 4
    p.x_dtype, p.weight_dtype = nat.GDN_BF16, nat.GDN_F32
    p.x, p.output, p.doutput, p.dx = far(1), far(2), far(3), far(4)
    p.weight, p.dweight, p.cu_seqlens = far(5), far(6), far(7)
    if mode == 2:
        p.total_tokens, p.cu_seqlens = 3, None
    for f, v in kw.items():
        setattr(p, f, v)
    return p


def _check_conv(p, mode=0, workspace=True):
    L = nat.lib()
    if workspace:
        p.workspace = ctypes.c_void_p(0x10000)
        p.workspace_bytes = L.gdn_convolution_workspace_size(ctypes.byref(p), int(mode == 1))
    return L.gdn_validate_convolution_host(ctypes.byref(p), mode)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_convolution_accepted(mode):
    for kw in (dict(), dict(x_dtype=nat.GDN_F32), dict(weight_dtype=nat.GDN_BF16), dict(width=2),
               dict(channels=1), dict(x_stride=100), dict(bias=FAKE), dict(silu=1),
               dict(initial_state=FAKE, initial_state_dtype=nat.GDN_FP8_E4M3),
               dict(x=ctypes.c_void_p(0x1002))):
        assert _check_conv(_conv(mode, **kw), mode) == 0, kw


@pytest.mark.parametrize("mode,kw,err", [
    (0, dict(width=1), "SHAPE"), (0, dict(width=5), "SHAPE"), (0, dict(channels=0), "SHAPE"),
    (0, dict(total_tokens=-1), "SHAPE"), (0, dict(cu_seqlens=None), "SHAPE"), (0, dict(silu=2), "SHAPE"),
    (0, dict(num_seqs=2 ** 30 + 1), "SHAPE"), (0, dict(total_tokens=2 ** 31 - 1), "SHAPE"),
    (0, dict(total_tokens=2 ** 30, channels=2 ** 20), "SHAPE"), (2, dict(total_tokens=4), "SHAPE"),
    (2, dict(total_tokens=2 ** 24, num_seqs=2 ** 24, channels=1), "SHAPE"),
    (2, dict(total_tokens=2 ** 23, num_seqs=2 ** 23, channels=257), "SHAPE"),
    (2, dict(cu_seqlens=FAKE), "SHAPE"), (0, dict(x_dtype=3), "DTYPE"),
    (0, dict(weight_dtype=nat.GDN_F16), "DTYPE"), (0, dict(cu_seqlens_type=5), "DTYPE"),
    (0, dict(x=None), "NULL"), (0, dict(weight=None), "NULL"), (0, dict(output=None), "NULL"),
    (1, dict(doutput=None), "NULL"), (1, dict(dx=None), "NULL"), (1, dict(dweight=None), "NULL"),
    (0, dict(x_stride=95), "STRIDES"), (1, dict(doutput_stride=7), "STRIDES"),
    (0, dict(x=ctypes.c_void_p(0x1001)), "ALIGN"), (0, dict(weight=ctypes.c_void_p(0x1002)), "ALIGN"),
    (1, dict(dweight=ctypes.c_void_p(0x1002)), "ALIGN"), (0, dict(output=far(1)), "STATE"),
    (0, dict(output=ctypes.c_void_p(far(1).value + 100)), "STATE"), (1, dict(dx=far(3)), "STATE"),
    (1, dict(dx=far(1)), "STATE"), (1, dict(state_indices=FAKE, pool_size=4), "STATE"),
    (0, dict(state_indices=FAKE), "STATE"), (0, dict(output_final_state=1), "STATE"),
    (0, dict(initial_state=FAKE, initial_state_dtype=9), "DTYPE"),
    (0, dict(initial_state=FAKE, initial_state_stride=287), "STRIDES")])
def test_convolution_refused(mode, kw, err):
    assert _check_conv(_conv(mode, **kw), mode) == code("GDN_ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    # the same rows: every thread reads what it overwrites
    (dict(output=far(1)), None), (dict(output=far(1), x_stride=96), None),
    (dict(output=far(1), x_stride=100, total_tokens=1, num_seqs=1), None),
    # a row or a channel further on, or rows at another distance
    (dict(output=ctypes.c_void_p(far(1).value + 2)), "STATE"),
    (dict(output=ctypes.c_void_p(far(1).value + 192)), "STATE"),
    (dict(output=far(1), x_stride=100), "STATE"),
    (dict(output=ctypes.c_void_p(far(1).value + 3 * 192)), None),
    (dict(output=ctypes.c_void_p(far(1).value + 2), total_tokens=1, num_seqs=1), "STATE")])
def test_convolution_decode_in_place(kw, err):
    assert _check_conv(_conv(2, **kw), 2) == (code("GDN_ERR_" + err) if err else 0)


def test_convolution_workspace():
    L = nat.lib()
    assert L.gdn_convolution_workspace_size(ctypes.byref(_conv()), 0) == 0
    p = _conv(num_seqs=64)
    assert L.gdn_convolution_workspace_size(ctypes.byref(p), 0) >= 4 * 65
    assert _check_conv(p, 0, workspace=False) == code("GDN_ERR_WORKSPACE")
    q = _conv(1)
    need = L.gdn_convolution_workspace_size(ctypes.byref(q), 1)
    # the size depends on the sizes alone
    for kw in (dict(x=None), dict(x=ctypes.c_void_p(0x1002)), dict(doutput_stride=97)):
        assert L.gdn_convolution_workspace_size(ctypes.byref(_conv(1, **kw)), 1) == need
    q.workspace, q.workspace_bytes = ctypes.c_void_p(0x10000), need - 1
    assert _check_conv(q, 1, workspace=False) == code("GDN_ERR_WORKSPACE")
    q.workspace, q.workspace_bytes = ctypes.c_void_p(0x10010), need
    assert _check_conv(q, 1, workspace=False) == code("GDN_ERR_ALIGN")


# ----------------------------------------------------------------------- scan

def _scan(mode=0, **kw):
    p = nat.ScanParams()
    p.total_tokens, p.num_seqs, p.channels, p.num_states, p.groups = 1000, 3, 96, 16, 2
    p.x_dtype = nat.GDN_BF16
    for k, f in enumerate(("x", "delta", "B", "C", "output", "doutput", "dx", "ddelta", "dB", "dC",
                           "A", "dA", "cu_seqlens")):
        setattr(p, f, far(k + 1))
    if mode == 2:
        p.total_tokens, p.cu_seqlens = 3, None
    for f, v in kw.items():
        setattr(p, f, v)
    return p


def _check_scan(p, mode=0, workspace=True):
    L = nat.lib()
    if workspace:
        p.workspace = ctypes.c_void_p(0x10000)
        p.workspace_bytes = L.gdn_scan_workspace_size(ctypes.byref(p), int(mode == 1))
    return L.gdn_validate_scan_host(ctypes.byref(p), mode)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_scan_accepted(mode):
    for kw in (dict(), dict(x_dtype=nat.GDN_F32), dict(num_states=1), dict(num_states=64),
               dict(groups=96), dict(x_stride=100, b_stride=33), dict(D=FAKE, delta_bias=FAKE),
               dict(z=far(20), dz=far(21)), dict(delta_softplus=1),
               dict(initial_state=FAKE, initial_state_dtype=nat.GDN_F32)):
        assert _check_scan(_scan(mode, **kw), mode) == 0, kw


@pytest.mark.parametrize("mode,kw,err", [
    (0, dict(num_states=0), "SHAPE"), (0, dict(num_states=65), "SHAPE"), (0, dict(groups=5), "SHAPE"),
    (0, dict(groups=0), "SHAPE"), (0, dict(channels=2 ** 24 + 2), "SHAPE"),
    (0, dict(total_tokens=2 ** 30, channels=2 ** 20), "SHAPE"), (0, dict(cu_seqlens=None), "SHAPE"),
    (0, dict(delta_softplus=2), "SHAPE"), (2, dict(total_tokens=4), "SHAPE"),
    (2, dict(total_tokens=2 ** 29, num_seqs=2 ** 29), "SHAPE"), (0, dict(x_dtype=4), "DTYPE"),
    (2, dict(total_tokens=2 ** 24, num_seqs=2 ** 24, channels=1, groups=1), "SHAPE"),
    (2, dict(total_tokens=2 ** 22, num_seqs=2 ** 22, channels=65, groups=1, num_states=64), "SHAPE"),
    (0, dict(A=None), "NULL"), (0, dict(delta=None), "NULL"), (0, dict(B=None), "NULL"),
    (1, dict(dA=None), "NULL"), (1, dict(dC=None), "NULL"), (1, dict(z=far(20)), "NULL"),
    (0, dict(delta_stride=95), "STRIDES"), (0, dict(c_stride=31), "STRIDES"),
    (0, dict(B=ctypes.c_void_p(0x1001)), "ALIGN"), (0, dict(A=ctypes.c_void_p(0x1002)), "ALIGN"),
    (0, dict(output=far(1)), "STATE"), (0, dict(output=far(3)), "STATE"), (1, dict(dx=far(2)), "STATE"),
    (2, dict(chunk_states=FAKE), "STATE"), (1, dict(state_indices=FAKE, pool_size=3), "STATE"),
    (1, dict(initial_state=FAKE, initial_state_dtype=nat.GDN_BF16), "DTYPE"),
    (0, dict(initial_state=FAKE, initial_state_stride=5), "STRIDES")])
def test_scan_refused(mode, kw, err):
    assert _check_scan(_scan(mode, **kw), mode) == code("GDN_ERR_" + err)


@pytest.mark.parametrize("out", ["dx", "ddelta", "dz", "dB", "dC"])
def test_scan_gradients_over_doutput(out):
    """Tokens of the gradient of the output are read by several workgroups."""
    kw = dict(z=far(20), dz=far(21))
    last = far(6).value + 2 * (1000 * 96 - 1)
    assert _check_scan(_scan(1, **dict(kw, **{out: far(6)})), 1) == code("GDN_ERR_STATE")
    assert _check_scan(_scan(1, **dict(kw, **{out: ctypes.c_void_p(last)})), 1) == code("GDN_ERR_STATE")
    assert _check_scan(_scan(1, **dict(kw, **{out: ctypes.c_void_p(last + 2)})), 1) == 0
    assert _check_scan(_scan(0, doutput=far(5)), 0) == 0  # not looked at


def test_scan_workspace_and_chunk():
    L = nat.lib()
    p = _scan()
    assert L.gdn_scan_chunk(ctypes.byref(p)) == 16
    for n, most in ((16, 64), (8, 64), (32, 32), (64, 16)):
        big = _scan(total_tokens=1 << 20, channels=4096, groups=1, num_states=n)
        assert L.gdn_scan_chunk(ctypes.byref(big)) == most
    assert L.gdn_scan_chunk(ctypes.byref(_scan(groups=5))) == 0
    need = L.gdn_scan_workspace_size(ctypes.byref(p), 0)
    p.workspace, p.workspace_bytes = ctypes.c_void_p(0x10000), need - 1
    assert _check_scan(p, 0, workspace=False) == code("GDN_ERR_WORKSPACE")
    # states that the caller keeps are not in the workspace
    q = _scan(1)
    own = L.gdn_scan_workspace_size(ctypes.byref(q), 1)
    q.chunk_states = FAKE
    assert L.gdn_scan_workspace_size(ctypes.byref(q), 1) < own
    assert _check_scan(_scan(total_tokens=0, x=None, delta=None, B=None, C=None, output=None)) == 0


@pytest.mark.parametrize("width,channels,ok", [
    (4, 107374176, True), (4, 107374177, False), (2, 178956960, True), (2, 178956961, False)])
def test_convolution_backward_grid(width, channels, ok):
    """The sums over tokens: fewer than 2^24 workgroups of 32 columns."""
    kw = dict(width=width, channels=channels, total_tokens=0, num_seqs=0, x=None, doutput=None, dx=None)
    assert _check_conv(_conv(1, **kw), 1) == (0 if ok else code("GDN_ERR_SHAPE"))
    assert _check_conv(_conv(0, **dict(kw, output=None)), 0) == 0


@pytest.mark.parametrize("states,channels,ok", [
    (64, 8134407, True), (64, 8134408, False), (30, 2 ** 24 - 1, True), (30, 2 ** 24, False)])
def test_scan_backward_grid_without_tokens(states, channels, ok):
    kw = dict(num_states=states, channels=channels, groups=1, total_tokens=0)
    assert _check_scan(_scan(1, **kw), 1) == (0 if ok else code("GDN_ERR_SHAPE"))
    assert _check_scan(_scan(0, **kw), 0) == 0


# ----------------------------------------------------------------------- beam

def _beam(**kw):
    p = nat.BeamParams()
    p.num_groups, p.num_beams, p.vocab, p.num_candidates = 2, 4, 1000, 8
    p.logits = p.scores = p.out_scores = p.out_parents = p.out_tokens = FAKE
    for f, v in kw.items():
        setattr(p, f, v)
    p.workspace = ctypes.c_void_p(0x10000)
    p.workspace_bytes = nat.lib().gdn_beam_workspace_size(ctypes.byref(p))
    return p


@pytest.mark.parametrize("kw,err", [
    (dict(), None), (dict(logits_dtype=nat.GDN_F16, logits_stride=1001), None), (dict(num_groups=0), None),
    (dict(num_beams=0), "SHAPE"), (dict(num_beams=65), "SHAPE"), (dict(num_candidates=0), "SHAPE"),
    (dict(num_candidates=65), "SHAPE"), (dict(vocab=0), "SHAPE"), (dict(vocab=2 ** 28 + 1), "SHAPE"),
    (dict(vocab=1, num_candidates=5), "SHAPE"), (dict(num_groups=2 ** 24), "SHAPE"),
    (dict(logits_dtype=3), "DTYPE"), (dict(logits_stride=999), "STRIDES"), (dict(scores=None), "NULL"),
    (dict(out_tokens=None), "NULL"), (dict(logits=ctypes.c_void_p(0x1002)), "ALIGN")])
def test_beam(kw, err):
    got = nat.lib().gdn_validate_beam_host(ctypes.byref(_beam(**kw)))
    assert got == (code("GDN_ERR_" + err) if err else 0)


def test_beam_workspace():
    p = _beam()
    p.workspace_bytes -= 1
    assert nat.lib().gdn_validate_beam_host(ctypes.byref(p)) == code("GDN_ERR_WORKSPACE")


def _reorder(pool=None, **kw):
    q = nat.ReorderPool()
    q.pool, q.dtype = FAKE, nat.GDN_F32
    q.extent[:] = [2, 3, 4]
    for f, v in (pool or {}).items():
        if f in ("extent", "strides"):
            getattr(q, f)[:] = v
        else:
            setattr(q, f, v)
    p = nat.ReorderParams()
    p.num_groups, p.num_beams, p.num_pools, p.pool_rows = 2, 4, 1, 9
    p.pools = ctypes.cast(ctypes.byref(q), ctypes.c_void_p)
    p.state_indices, p.parents, p.new_indices = far(1), far(2), far(3)
    for f, v in kw.items():
        setattr(p, f, v)
    return nat.lib().gdn_validate_reorder_host(ctypes.byref(p))


@pytest.mark.parametrize("pool,kw,err", [
    ({}, {}, None), (dict(strides=[30, 12, 4, 1]), {}, None), ({}, dict(num_groups=0, pool_rows=0), None),
    ({}, dict(num_beams=65), "SHAPE"), ({}, dict(num_pools=0), "SHAPE"), ({}, dict(pool_rows=262145), "SHAPE"),
    ({}, dict(num_groups=2 ** 17), "SHAPE"), (dict(extent=[0, 1, 1]), {}, "SHAPE"),
    (dict(dtype=9), {}, "DTYPE"), ({}, dict(index_type=2), "DTYPE"), (dict(pool=None), {}, "NULL"),
    ({}, dict(parents=None), "NULL"), ({}, dict(new_indices=far(1)), "STATE"),
    ({}, dict(new_indices=ctypes.c_void_p(far(2).value + 28)), "STATE"), ({}, dict(pool_rows=0), "STATE"),
    (dict(pool=ctypes.c_void_p(0x1002)), {}, "ALIGN"), (dict(strides=[20, 12, 4, 1]), {}, "STRIDES"),
    (dict(strides=[24, 12, 4, 0]), {}, "STRIDES")])
def test_reorder(pool, kw, err):
    assert _reorder(pool, **kw) == (code("GDN_ERR_" + err) if err else 0)


BASE = 0x10000000


def _view(at, extent, strides=(0, 0, 0, 0), dtype=nat.GDN_F32):
    return (BASE + at, dtype, list(extent), list(strides))


def _reorder_of(views, rows):
    pools = (nat.ReorderPool * len(views))()
    for q, (at, dtype, extent, strides) in zip(pools, views):
        q.pool, q.dtype = ctypes.c_void_p(at), dtype
        q.extent[:], q.strides[:] = extent, strides
    p = nat.ReorderParams()
    p.num_groups, p.num_beams, p.num_pools, p.pool_rows = 2, 4, len(views), rows
    p.pools = ctypes.cast(pools, ctypes.c_void_p)
    p.state_indices, p.parents, p.new_indices = far(1), far(2), far(3)
    return nat.lib().gdn_validate_reorder_host(ctypes.byref(p))


LAYERS = [_view(4 * 132 * i, (1, 4, 33), (9 * 132, 1, 33, 1)) for i in range(9)]


@pytest.mark.parametrize("views", [
    # one after the other; the layers of one [rows, layers, ...] buffer, in any order
    [_view(0, (2, 3, 4)), _view(4 * 24 * 20, (2, 3, 4))], LAYERS, LAYERS[::-1],
    LAYERS + [_view(4 * 9 * 132 * 20, (5, 1, 1))],
    # two kinds of states in one buffer of 100 elements a row
    [_view(0, (1, 3, 20), (100, 1, 20, 1)), _view(240, (1, 4, 10), (100, 1, 10, 1))],
    [_view(0, (1, 3, 20), (100, 1, 20, 1)), _view(240, (1, 4, 20), (200, 1, 20, 1), nat.GDN_BF16)],
    # rows apart in one period, the second view's begin behind the first's end
    [_view(4 * 100, (1, 1, 60), (100, 1, 1, 1)), _view(240, (1, 1, 40), (100, 1, 1, 1))],
    # interleaved closer than row by row: alternate heads, layers in front of the rows
    [_view(0, (4, 1, 10), (100, 20, 1, 1)), _view(40, (4, 1, 10), (100, 20, 1, 1))],
    [_view(0, (3, 1, 6), (6, 240, 1, 1)), _view(4 * 120, (3, 1, 6), (6, 240, 1, 1))],
])
def test_reorder_of_pools_that_are_apart(views):
    assert _reorder_of(views, 20) == 0


@pytest.mark.parametrize("views", [
    # the same one twice; a row or an element further on; a part of a row; as another type
    [_view(0, (2, 3, 4)), _view(0, (2, 3, 4))], [_view(0, (2, 3, 4)), _view(96, (2, 3, 4))],
    [_view(0, (2, 3, 4)), _view(4, (2, 3, 4))],
    [_view(0, (2, 3, 4)), _view(8, (1, 1, 4), (24, 1, 1, 1))],
    [_view(0, (2, 3, 4)), _view(0, (2, 3, 4), dtype=nat.GDN_F16)],
    [_view(0, (2, 3, 4)), _view(4 * 24 * 20 - 4, (1, 1, 1))],
    # one among many that are apart; rows that meet only across the period's end
    LAYERS + [_view(4 * (132 * 4 + 131), (1, 1, 2), (9 * 132, 1, 1, 1))], LAYERS[:5] + LAYERS[4:],
    [_view(0, (1, 1, 60), (100, 1, 1, 1)), _view(4 * 70, (1, 1, 40), (100, 1, 1, 1))],
    [_view(0, (4, 1, 10), (100, 20, 1, 1)), _view(36, (4, 1, 10), (100, 20, 1, 1))],
])
def test_reorder_of_pools_that_share_elements(views):
    assert _reorder_of(views, 20) == code("GDN_ERR_STATE")


def test_null_blocks():
    L = nat.lib()
    null = code("GDN_ERR_NULL")
    for f in (L.gdn_convolution, L.gdn_convolution_backward, L.gdn_convolution_decode, L.gdn_scan,
              L.gdn_scan_backward, L.gdn_scan_decode, L.gdn_beam_select, L.gdn_pool_reorder):
        assert f(None, None) == null
    for f in (L.gdn_validate_convolution_host, L.gdn_validate_scan_host):
        assert f(None, 0) == null
    assert L.gdn_validate_convolution_host(ctypes.byref(_conv()), 3) == code("GDN_ERR_SHAPE")
    assert L.gdn_validate_scan_host(ctypes.byref(_scan()), -1) == code("GDN_ERR_SHAPE")


def test_python_calls_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import gated_deltanet_chunked_varlen_amd as gdn
    x, w = torch.zeros((4, 8)), torch.zeros((8, 4))
    A, B = torch.zeros((8, 4)), torch.zeros((4, 1, 4))
    idx, par = torch.zeros(2, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    for call in (lambda: gdn.short_convolution(x, w), lambda: gdn.short_convolution_backward(x, x, w),
                 lambda: gdn.short_convolution_decode(x, w), lambda: gdn.short_convolution(x, w, activation="gelu"),
                 lambda: gdn.selective_scan(x, x, A, B, B),
                 lambda: gdn.selective_scan_backward(x, x, x, A, B, B),
                 lambda: gdn.selective_scan_decode(x, x, A, B, B),
                 lambda: gdn.beam_select(x[None], x[:1, :4]), lambda: gdn.state_pool_reorder(x, idx, par),
                 lambda: gdn.state_pool_reorder([], idx, par), lambda: gdn.short_convolution(3, w),
                 lambda: gdn.short_convolution(x.requires_grad_(), w, output=x)):
        with pytest.raises(ValueError):
            call()
