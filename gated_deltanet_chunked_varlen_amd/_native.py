"""ctypes view of libgdn_prefill (include/gdn_prefill.h).

Argument marshalling only: no arithmetic of the method happens in Python.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_PREFILL_LIB names another build of the library (e.g. one whose host
# code carries sanitizers); the default is the in-tree build
LIB_PATH = os.environ.get("GDN_PREFILL_LIB") or os.path.join(HERE, "libgdn_prefill.so")

GDN_F32, GDN_BF16, GDN_F16, GDN_FP8_E4M3, GDN_FP8_E5M2 = 0, 1, 2, 3, 4
GDN_I32, GDN_I64 = 0, 1

GDN_OK = 0
ERRORS = {
    -1: "GDN_ERR_NULL", -2: "GDN_ERR_SHAPE", -3: "GDN_ERR_HEAD_RATIO",
    -4: "GDN_ERR_DTYPE", -5: "GDN_ERR_CHECKPOINT", -6: "GDN_ERR_STATE",
    -7: "GDN_ERR_MAX_SEQLEN", -8: "GDN_ERR_WORKSPACE", -9: "GDN_ERR_STRIDES",
    -10: "GDN_ERR_DEVICE", -11: "GDN_ERR_LAUNCH", -12: "GDN_ERR_ALIGN",
    -13: "GDN_ERR_SCRATCH", -14: "GDN_ERR_CP",
}
NOALLOC_SCRATCH_BYTES = 128 << 20
CP_AUTO, CP_ON, CP_OFF = 0, 1, 2
ABI_VERSION = 2
ERR_CODE = {v: k for k, v in ERRORS.items()}
STATUS_CU_SEQLENS = 1
STATUS_CHECKPOINT_STARTS = 2
STATUS_STATE_INDEX = 4
STATUS_CHUNK_CAPACITY = 8
STATUS_POOL_ROW = 16
STATUS_POOL_DUPLICATE = 32
STATUS_POOL_OVERLAP = 64
RECURRENCE_CHUNK = 64
POOL_MAX_ROWS = 262144
BEAM_MAX = 64

# every symbol include/gdn_prefill.h declares
EXPORTS = [
    "gdn_abi_version", "gdn_status_string", "gdn_max_chunks",
    "gdn_prefill_workspace_size", "gdn_validate_host", "gdn_prefill",
    "gdn_prefill_timed", "gdn_build_chunk_indices", "gdn_decode",
    "gdn_validate_decode_host", "gdn_prefill_noalloc",
    "gdn_recurrence_workspace_size", "gdn_validate_recurrence_host", "gdn_recurrence",
    "gdn_recurrence_backward", "gdn_recurrence_decode", "gdn_validate_pool_host",
    "gdn_pool_copy", "gdn_pool_reset", "gdn_pool_compact",
    "gdn_convolution_workspace_size", "gdn_validate_convolution_host", "gdn_convolution",
    "gdn_convolution_backward", "gdn_convolution_decode",
    "gdn_scan_chunk", "gdn_scan_workspace_size", "gdn_validate_scan_host", "gdn_scan",
    "gdn_scan_backward", "gdn_scan_decode",
    "gdn_beam_workspace_size", "gdn_validate_beam_host", "gdn_beam_select",
    "gdn_validate_reorder_host", "gdn_pool_reorder",
]

_i64x4 = ctypes.c_int64 * 4


class Params(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_k_heads", ctypes.c_int32),
        ("num_v_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("qkv_dtype", ctypes.c_int32),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("beta", ctypes.c_void_p),
        ("has_scale", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("cu_seqlens", ctypes.c_void_p),
        ("cu_seqlens_type", ctypes.c_int32),
        ("use_qk_l2norm_in_kernel", ctypes.c_int32),
        ("output", ctypes.c_void_p),
        ("initial_state", ctypes.c_void_p),
        ("initial_state_dtype", ctypes.c_int32),
        ("initial_state_strides", _i64x4),
        ("output_final_state", ctypes.c_int32),
        ("output_state", ctypes.c_void_p),
        ("output_state_dtype", ctypes.c_int32),
        ("output_state_strides", _i64x4),
        ("state_indices", ctypes.c_void_p),
        ("state_indices_type", ctypes.c_int32),
        ("pool_size", ctypes.c_int64),
        ("checkpoint_every_n_tokens", ctypes.c_int32),
        ("state_checkpoints", ctypes.c_void_p),
        ("checkpoint_dtype", ctypes.c_int32),
        ("checkpoint_rows", ctypes.c_int64),
        ("checkpoint_cu_starts", ctypes.c_void_p),
        ("checkpoint_cu_starts_type", ctypes.c_int32),
        ("max_seqlen", ctypes.c_int64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
        ("use_cp", ctypes.c_int32),
        ("cp_chunk_len", ctypes.c_int64),
    ]


class RecurrenceParams(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("g_dtype", ctypes.c_int32),
        ("g_per_head", ctypes.c_int32),
        ("x", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("g_stride", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p),
        ("cu_seqlens_type", ctypes.c_int32),
        ("output", ctypes.c_void_p),
        ("initial_state", ctypes.c_void_p),
        ("initial_state_dtype", ctypes.c_int32),
        ("initial_state_stride", ctypes.c_int64),
        ("output_final_state", ctypes.c_int32),
        ("output_state", ctypes.c_void_p),
        ("output_state_dtype", ctypes.c_int32),
        ("output_state_stride", ctypes.c_int64),
        ("state_indices", ctypes.c_void_p),
        ("state_indices_type", ctypes.c_int32),
        ("pool_size", ctypes.c_int64),
        ("chunk_states", ctypes.c_void_p),
        ("doutput", ctypes.c_void_p),
        ("doutput_stride", ctypes.c_int64),
        ("dfinal_state", ctypes.c_void_p),
        ("dx", ctypes.c_void_p),
        ("dg", ctypes.c_void_p),
        ("dinitial_state", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


_i64x3 = ctypes.c_int64 * 3


class PoolParams(ctypes.Structure):
    _fields_ = [
        ("extent", _i64x3),
        ("src", ctypes.c_void_p),
        ("src_dtype", ctypes.c_int32),
        ("src_pool_rows", ctypes.c_int64),
        ("src_strides", _i64x4),
        ("dst", ctypes.c_void_p),
        ("dst_dtype", ctypes.c_int32),
        ("dst_pool_rows", ctypes.c_int64),
        ("dst_strides", _i64x4),
        ("src_rows", ctypes.c_void_p),
        ("dst_rows", ctypes.c_void_p),
        ("rows_type", ctypes.c_int32),
        ("count", ctypes.c_int64),
        ("status", ctypes.c_void_p),
    ]


class ConvolutionParams(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("silu", ctypes.c_int32),
        ("x", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("weight", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p),
        ("cu_seqlens_type", ctypes.c_int32),
        ("output", ctypes.c_void_p),
        ("initial_state", ctypes.c_void_p),
        ("initial_state_dtype", ctypes.c_int32),
        ("initial_state_stride", ctypes.c_int64),
        ("output_final_state", ctypes.c_int32),
        ("output_state", ctypes.c_void_p),
        ("output_state_dtype", ctypes.c_int32),
        ("output_state_stride", ctypes.c_int64),
        ("state_indices", ctypes.c_void_p),
        ("state_indices_type", ctypes.c_int32),
        ("pool_size", ctypes.c_int64),
        ("doutput", ctypes.c_void_p),
        ("doutput_stride", ctypes.c_int64),
        ("dfinal_state", ctypes.c_void_p),
        ("dx", ctypes.c_void_p),
        ("dweight", ctypes.c_void_p),
        ("dbias", ctypes.c_void_p),
        ("dinitial_state", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


class ScanParams(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("num_states", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("delta_softplus", ctypes.c_int32),
        ("x", ctypes.c_void_p),
        ("delta", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("delta_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64),
        ("A", ctypes.c_void_p),
        ("B", ctypes.c_void_p),
        ("C", ctypes.c_void_p),
        ("b_stride", ctypes.c_int64),
        ("c_stride", ctypes.c_int64),
        ("D", ctypes.c_void_p),
        ("delta_bias", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p),
        ("cu_seqlens_type", ctypes.c_int32),
        ("output", ctypes.c_void_p),
        ("initial_state", ctypes.c_void_p),
        ("initial_state_dtype", ctypes.c_int32),
        ("initial_state_stride", ctypes.c_int64),
        ("output_final_state", ctypes.c_int32),
        ("output_state", ctypes.c_void_p),
        ("output_state_dtype", ctypes.c_int32),
        ("output_state_stride", ctypes.c_int64),
        ("state_indices", ctypes.c_void_p),
        ("state_indices_type", ctypes.c_int32),
        ("pool_size", ctypes.c_int64),
        ("chunk_states", ctypes.c_void_p),
        ("doutput", ctypes.c_void_p),
        ("doutput_stride", ctypes.c_int64),
        ("dfinal_state", ctypes.c_void_p),
        ("dx", ctypes.c_void_p),
        ("ddelta", ctypes.c_void_p),
        ("dz", ctypes.c_void_p),
        ("dB", ctypes.c_void_p),
        ("dC", ctypes.c_void_p),
        ("dA", ctypes.c_void_p),
        ("dD", ctypes.c_void_p),
        ("ddelta_bias", ctypes.c_void_p),
        ("dinitial_state", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


class BeamParams(ctypes.Structure):
    _fields_ = [
        ("num_groups", ctypes.c_int32),
        ("num_beams", ctypes.c_int32),
        ("vocab", ctypes.c_int32),
        ("num_candidates", ctypes.c_int32),
        ("logits_dtype", ctypes.c_int32),
        ("logits", ctypes.c_void_p),
        ("logits_stride", ctypes.c_int64),
        ("scores", ctypes.c_void_p),
        ("out_scores", ctypes.c_void_p),
        ("out_parents", ctypes.c_void_p),
        ("out_tokens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class ReorderPool(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("extent", _i64x3),
        ("strides", _i64x4),
    ]


class ReorderParams(ctypes.Structure):
    _fields_ = [
        ("num_groups", ctypes.c_int32),
        ("num_beams", ctypes.c_int32),
        ("num_pools", ctypes.c_int32),
        ("pool_rows", ctypes.c_int64),
        ("pools", ctypes.c_void_p),
        ("state_indices", ctypes.c_void_p),
        ("parents", ctypes.c_void_p),
        ("new_indices", ctypes.c_void_p),
        ("index_type", ctypes.c_int32),
        ("status", ctypes.c_void_p),
    ]

_lib = None


def lib():
    """Load the in-tree library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libgdn_prefill.so is not built; run "
                "`python -m gated_deltanet_chunked_varlen_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.gdn_abi_version.restype = ctypes.c_int
        L.gdn_abi_version.argtypes = []
        if L.gdn_abi_version() != ABI_VERSION:
            raise ImportError("libgdn_prefill.so has ABI version %d, this binding expects %d; "
                              "rebuild it" % (L.gdn_abi_version(), ABI_VERSION))
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_max_chunks.restype = ctypes.c_int64
        L.gdn_max_chunks.argtypes = [ctypes.c_int64, ctypes.c_int32]
        L.gdn_prefill_workspace_size.restype = ctypes.c_size_t
        L.gdn_prefill_workspace_size.argtypes = [ctypes.POINTER(Params)]
        L.gdn_validate_host.restype = ctypes.c_int
        L.gdn_validate_host.argtypes = [ctypes.POINTER(Params)]
        L.gdn_prefill.restype = ctypes.c_int
        L.gdn_prefill.argtypes = [ctypes.POINTER(Params), ctypes.c_void_p]
        L.gdn_prefill_timed.restype = ctypes.c_int
        L.gdn_prefill_timed.argtypes = [ctypes.POINTER(Params), ctypes.c_void_p,
                                        ctypes.c_void_p * 5]
        L.gdn_prefill_noalloc.restype = ctypes.c_int
        L.gdn_prefill_noalloc.argtypes = [ctypes.POINTER(Params), ctypes.c_void_p]
        L.gdn_decode.restype = ctypes.c_int
        L.gdn_decode.argtypes = [ctypes.POINTER(Params), ctypes.c_void_p]
        L.gdn_validate_decode_host.restype = ctypes.c_int
        L.gdn_validate_decode_host.argtypes = [ctypes.POINTER(Params)]
        L.gdn_build_chunk_indices.restype = ctypes.c_int
        L.gdn_build_chunk_indices.argtypes = [
            ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        rec, pool = ctypes.POINTER(RecurrenceParams), ctypes.POINTER(PoolParams)
        L.gdn_recurrence_workspace_size.restype = ctypes.c_size_t
        L.gdn_recurrence_workspace_size.argtypes = [rec, ctypes.c_int32]
        L.gdn_validate_recurrence_host.restype = ctypes.c_int
        L.gdn_validate_recurrence_host.argtypes = [rec, ctypes.c_int32]
        for name in ("gdn_recurrence", "gdn_recurrence_backward", "gdn_recurrence_decode"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [rec, ctypes.c_void_p]
        L.gdn_validate_pool_host.restype = ctypes.c_int
        L.gdn_validate_pool_host.argtypes = [pool, ctypes.c_int32]
        for name in ("gdn_pool_copy", "gdn_pool_reset"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [pool, ctypes.c_void_p]
        L.gdn_pool_compact.restype = ctypes.c_int
        L.gdn_pool_compact.argtypes = [pool, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p]
        for what, cls in (("convolution", ConvolutionParams), ("scan", ScanParams)):
            block = ctypes.POINTER(cls)
            size = getattr(L, "gdn_%s_workspace_size" % what)
            size.restype, size.argtypes = ctypes.c_size_t, [block, ctypes.c_int32]
            check = getattr(L, "gdn_validate_%s_host" % what)
            check.restype, check.argtypes = ctypes.c_int, [block, ctypes.c_int32]
            for name in ("gdn_%s", "gdn_%s_backward", "gdn_%s_decode"):
                getattr(L, name % what).restype = ctypes.c_int
                getattr(L, name % what).argtypes = [block, ctypes.c_void_p]
        L.gdn_scan_chunk.restype = ctypes.c_int64
        L.gdn_scan_chunk.argtypes = [ctypes.POINTER(ScanParams)]
        beam, order = ctypes.POINTER(BeamParams), ctypes.POINTER(ReorderParams)
        L.gdn_beam_workspace_size.restype = ctypes.c_size_t
        L.gdn_beam_workspace_size.argtypes = [beam]
        for name, block in (("gdn_validate_beam_host", beam), ("gdn_validate_reorder_host", order)):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [block]
        for name, block in (("gdn_beam_select", beam), ("gdn_pool_reorder", order)):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [block, ctypes.c_void_p]
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().gdn_status_string(int(code)).decode()
