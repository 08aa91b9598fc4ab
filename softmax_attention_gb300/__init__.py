"""GB300 (sm_103a) fused softmax-attention forward: Python binding of libfa.so.

Argument marshalling only.  Every step of the computation runs in the CUDA kernels behind
the C ABI in ``include/fa.h``; PyTorch provides device memory and the current stream.  There
is no fallback: if the library is missing or a call fails, an exception is raised.

Entry points (same names as the C ABI):
    fa_prefill(q, k, v, causal, scale)                       bf16, spec signature
    fa_prefill_ex(q, k, v, causal=..., scale=..., mask=..., num_splits=..., dtype from q)
    fa_decode_paged(q, k_pages, v_pages, page_table, seq_lens, max_seq_len, scale)
    mla_decode_paged(q_nope, q_pe, ckv, kpe, page_table, seq_lens, max_seq_len, scale)
    fa_merge_states(o_parts, lse_parts, n_splits=None, out_dtype=torch.bfloat16)
    rotary_frequencies(rot_dim, base, scaling, factor, ...)  a table for the next two, on the host
    fa_rotary(q, k, positions, inv_freq, ...)                rotary positions (and their gradient)
    fa_cache_append(k, v, k_pages, v_pages, page_table, seq_lens, ...)   16-bit or e4m3 pages
    fa_cache_gather(k_pages, v_pages, page_table, seq_lens, max_seq_len, ...)
    tree_mask(parents)                                       a mask for the next one, on the host
    fa_tree_decode_paged(q, k_pages, v_pages, page_table, seq_lens, max_seq_len, tree_mask=...)
    fa_qk_norm_rotary(q, k, positions, inv_freq, q_weight, k_weight, ...)   and its _backward
    fa_prefill_packed(q, k, v, cu_seqlens_q, ...)            prompts behind one another, and its _backward
    gated_delta_step(q, k, v, g, beta, states, ...)          the gated delta rule token by token
    fa_get_device_status()
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE, FA_ERR_CUDA, FA_ERR_TIMEOUT, \
    FA_ERR_BOUNDS = range(7)
FA_BF16, FA_FP16, FA_FP32, FA_E4M3 = 0, 1, 2, 3
_DT = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16, torch.float32: FA_FP32}

# Every symbol include/fa.h declares.
EXPORTS = (
    "fa_prefill", "fa_prefill_ex", "fa_prefill_workspace_size", "fa_prefill_num_splits",
    "fa_prefill_paged", "fa_prefill_paged_workspace_size",
    "fa_decode_paged", "fa_decode_paged_ex", "fa_decode_workspace_size", "fa_decode_chunk_tokens",
    "fa_decode_get_plan",
    "fa_decode_paged_noalloc",
    "fa_decode_paged_states", "mla_decode_paged", "mla_decode_workspace_size",
    "mla_decode_chunk_tokens", "mla_decode_paged_states", "mla_decode_paged_ex", "fa_merge_states",
    "fa_get_device_status", "fa_selftest_wait_timeout", "fa_last_error", "fa_version",
    "gated_delta_prefill", "gated_delta_workspace_size",
    "fa_rotary", "fa_rotary_frequencies", "fa_cache_append", "fa_cache_gather",
    "fa_tree_decode_paged", "fa_tree_workspace_size", "fa_tree_mask",
    "fa_qk_norm_rotary", "fa_qk_norm_rotary_backward", "fa_qk_norm_rotary_backward_workspace_size",
    "fa_prefill_packed", "fa_packed_workspace_size",
    "fa_prefill_packed_backward", "fa_packed_backward_workspace_size",
    "gated_delta_step",
)


class FAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[fa status {code}] {msg}")
        self.code = code


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Lq", ctypes.c_int),
        ("Lkv", ctypes.c_int), ("D", ctypes.c_int), ("causal", ctypes.c_int),
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int), ("mask", ctypes.c_void_p),
        ("mask_dtype", ctypes.c_int), ("mask_batches", ctypes.c_int),
        ("num_splits", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
    ]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("max_seq_len", ctypes.c_int),
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("path", ctypes.c_int),
    ]


class DecodePlan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("n_splits", ctypes.c_int), ("launches", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t)]


# fa_decode_path
FA_DECODE_AUTO, FA_DECODE_CUDA_CORES, FA_DECODE_TENSOR_CORES = 0, 1, 2


class MlaArgs(ctypes.Structure):
    _fields_ = [
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("ckv_pages", ctypes.c_void_p), ("kpe_pages", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("Dc", ctypes.c_int), ("Dr", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("max_seq_len", ctypes.c_int),
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class GatedDeltaArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("initial_state", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("final_state", ctypes.c_void_p),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


_Strides = ctypes.c_int64 * 3


class RotaryArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p), ("q_strides", _Strides), ("k_strides", _Strides),
        ("q_out_strides", _Strides), ("k_out_strides", _Strides),
        ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
        ("D", ctypes.c_int), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
        ("transpose", ctypes.c_int), ("amplitude", ctypes.c_float), ("dtype", ctypes.c_int),
    ]


class CacheAppendArgs(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_strides", _Strides),
        ("v_strides", _Strides), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("inv_freq", ctypes.c_void_p),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float),
        ("dtype", ctypes.c_int), ("cache_dtype", ctypes.c_int),
    ]


class CacheGatherArgs(ctypes.Structure):
    _fields_ = [
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("max_seq_len", ctypes.c_int), ("dtype", ctypes.c_int), ("cache_dtype", ctypes.c_int),
    ]


class TreeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_strides", _Strides),
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("draft_lens", ctypes.c_void_p), ("tree_mask", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("T", ctypes.c_int),
        ("D", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("max_seq_len", ctypes.c_int),
        ("mask_batches", ctypes.c_int), ("num_splits", ctypes.c_int), ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int), ("cache_dtype", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


_Strides2 = ctypes.c_int64 * 2
_NORM_FIELDS = [
    ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
    ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
    ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
    ("D", ctypes.c_int), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
    ("amplitude", ctypes.c_float), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
    ("weight_dtype", ctypes.c_int),
]


class NormRotaryArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p), ("q_strides", _Strides), ("k_strides", _Strides),
        ("q_out_strides", _Strides), ("k_out_strides", _Strides),
    ] + _NORM_FIELDS


class NormRotaryBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("dq_out", ctypes.c_void_p), ("dk_out", ctypes.c_void_p), ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
        ("dq_weight", ctypes.c_void_p), ("dk_weight", ctypes.c_void_p),
        ("dq_out_strides", _Strides), ("dk_out_strides", _Strides), ("q_strides", _Strides),
        ("k_strides", _Strides), ("dq_strides", _Strides), ("dk_strides", _Strides),
    ] + _NORM_FIELDS + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_PACKED_FIELDS = [
    ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
    ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
    ("total_q", ctypes.c_int), ("total_k", ctypes.c_int), ("causal", ctypes.c_int),
    ("scale", ctypes.c_float), ("dtype", ctypes.c_int),
]


class PackedArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("q_strides", _Strides2), ("k_strides", _Strides2), ("v_strides", _Strides2),
        ("out_strides", _Strides2),
    ] + _PACKED_FIELDS + [("num_splits", ctypes.c_int), ("workspace", ctypes.c_void_p),
                          ("workspace_bytes", ctypes.c_size_t)]


class PackedBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("dout", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
        ("dout_strides", _Strides2), ("q_strides", _Strides2), ("k_strides", _Strides2),
        ("v_strides", _Strides2), ("out_strides", _Strides2), ("dq_strides", _Strides2),
        ("dk_strides", _Strides2), ("dv_strides", _Strides2),
    ] + _PACKED_FIELDS + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class GatedDeltaStepArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("states", ctypes.c_void_p),
        ("read_index", ctypes.c_void_p), ("write_index", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("q_strides", _Strides), ("k_strides", _Strides), ("v_strides", _Strides),
        ("g_strides", _Strides), ("beta_strides", _Strides), ("out_strides", _Strides),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("num_states", ctypes.c_int),
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int),
    ]


_lock = threading.Lock()
_lib = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_d = ctypes.c_double


def load_library(path: str | None = None):
    """Load libfa.so (built by ``softmax_attention_gb300.build``).  Raises if it is absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} not found: build it with `python -m softmax_attention_gb300.build`")
        lib = ctypes.CDLL(p)
        lib.fa_prefill.restype = _i
        lib.fa_prefill.argtypes = [_vp, _vp, _vp, _vp, _vp] + [_i] * 7 + [_f, _vp]
        lib.fa_prefill_ex.restype = _i
        lib.fa_prefill_ex.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
        lib.fa_prefill_workspace_size.restype = _sz
        lib.fa_prefill_workspace_size.argtypes = [ctypes.POINTER(PrefillArgs)]
        lib.fa_prefill_num_splits.restype = _i
        lib.fa_prefill_num_splits.argtypes = [ctypes.POINTER(PrefillArgs)]
        lib.fa_prefill_paged.restype = _i
        lib.fa_prefill_paged.argtypes = [_vp] * 7 + [_i] * 10 + [_f, _vp, _sz, _vp]
        lib.fa_prefill_paged_workspace_size.restype = _sz
        lib.fa_prefill_paged_workspace_size.argtypes = [_i] * 6
        lib.fa_decode_paged.restype = _i
        lib.fa_decode_paged.argtypes = [_vp] * 7 + [_i] * 8 + [_f, _vp, _sz, _vp]
        lib.fa_decode_paged_ex.restype = _i
        lib.fa_decode_paged_ex.argtypes = [ctypes.POINTER(DecodeArgs), _vp]
        lib.fa_decode_get_plan.restype = _i
        lib.fa_decode_get_plan.argtypes = [ctypes.POINTER(DecodeArgs), ctypes.POINTER(DecodePlan)]
        lib.mla_decode_paged_ex.restype = _i
        lib.mla_decode_paged_ex.argtypes = [ctypes.POINTER(MlaArgs), _vp]
        lib.fa_decode_workspace_size.restype = _sz
        lib.fa_decode_workspace_size.argtypes = [_i] * 4
        lib.fa_decode_paged_noalloc.restype = _i
        lib.fa_decode_paged_noalloc.argtypes = [_vp] * 7 + [_i] * 8 + [_f, _vp]
        lib.fa_decode_chunk_tokens.restype = _i
        lib.fa_decode_chunk_tokens.argtypes = [_i] * 3
        lib.fa_decode_paged_states.restype = _i
        lib.fa_decode_paged_states.argtypes = [_vp] * 7 + [_i] * 9 + [_f, _vp]
        lib.mla_decode_chunk_tokens.restype = _i
        lib.mla_decode_chunk_tokens.argtypes = [_i] * 3
        lib.mla_decode_paged_states.restype = _i
        lib.mla_decode_paged_states.argtypes = [_vp] * 8 + [_i] * 9 + [_f, _vp]
        lib.mla_decode_paged.restype = _i
        lib.mla_decode_paged.argtypes = [_vp] * 8 + [_i] * 8 + [_f, _vp, _sz, _vp]
        lib.mla_decode_workspace_size.restype = _sz
        lib.mla_decode_workspace_size.argtypes = [_i] * 4
        lib.fa_merge_states.restype = _i
        lib.fa_merge_states.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]
        lib.fa_get_device_status.restype = _i
        lib.fa_get_device_status.argtypes = [_vp]
        lib.fa_selftest_wait_timeout.restype = _i
        lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, _vp]
        lib.fa_last_error.restype = ctypes.c_char_p
        lib.fa_last_error.argtypes = []
        lib.fa_version.restype = _i
        lib.fa_version.argtypes = []
        lib.gated_delta_prefill.restype = _i
        lib.gated_delta_prefill.argtypes = [ctypes.POINTER(GatedDeltaArgs), _vp]
        lib.gated_delta_workspace_size.restype = _sz
        lib.gated_delta_workspace_size.argtypes = [ctypes.POINTER(GatedDeltaArgs)]
        lib.fa_rotary.restype = _i
        lib.fa_rotary.argtypes = [_vp, _vp]
        lib.fa_cache_append.restype = _i
        lib.fa_cache_append.argtypes = [_vp, _vp]
        lib.fa_cache_gather.restype = _i
        lib.fa_cache_gather.argtypes = [_vp, _vp]
        lib.fa_rotary_frequencies.restype = _i
        lib.fa_rotary_frequencies.argtypes = [_i, _d, _i, _d, _d, _d, _d, _vp, _vp]
        lib.fa_tree_mask.restype = _i
        lib.fa_tree_mask.argtypes = [_vp, _i, _vp]
        lib.fa_tree_decode_paged.restype = _i
        lib.fa_tree_decode_paged.argtypes = [_vp, _vp]
        lib.fa_tree_workspace_size.restype = _sz
        lib.fa_tree_workspace_size.argtypes = [_vp]
        for name in ("fa_qk_norm_rotary", "fa_qk_norm_rotary_backward", "fa_prefill_packed",
                     "fa_prefill_packed_backward", "gated_delta_step"):
            getattr(lib, name).restype = _i
            getattr(lib, name).argtypes = [_vp, _vp]
        for name in ("fa_qk_norm_rotary_backward_workspace_size", "fa_packed_workspace_size",
                     "fa_packed_backward_workspace_size"):
            getattr(lib, name).restype = _sz
            getattr(lib, name).argtypes = [_vp]
        _lib = lib
        return lib


def _check(rc: int):
    if rc != FA_OK:
        raise FAError(rc, load_library().fa_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_dtype(dtype, *ts):
    """The C entry points take raw pointers; element types are checked here."""
    for t in ts:
        if t is not None and t.dtype != dtype:
            raise ValueError(f"expected {dtype}, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _workspace(nbytes: int, device, workspace):
    if nbytes == 0:
        return None
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} bytes")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------------------------------
def fa_prefill(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
               stream=None):
    """bf16 dense attention through the short-form entry point (no KV split)."""
    lib = load_library()
    _need_dtype(torch.bfloat16, q, k, v, out)
    _need_dtype(torch.float32, lse)
    _need_cuda(q, k, v, out, lse)
    B, Hq, Lq, D = q.shape
    Hkv, Lkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, Lq, dtype=torch.float32, device=q.device)
    _check(lib.fa_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Lq, Lkv, D,
                          int(bool(causal)), float(scale), _stream(stream)))
    return out, lse


def prefill_args(q, k, v, *, causal=False, scale=None, out=None, lse=None, mask=None,
                 num_splits=0, workspace=None, page_table=None, seq_lens=None,
                 max_seq_len=None) -> PrefillArgs:
    """Argument struct of fa_prefill_ex.  Dense: k, v [B,Hkv,Lkv,D].  Paged (page_table
    given): k, v are pages [num_pages,Hkv,page_size,D] and Lkv = max_seq_len."""
    B, Hq, Lq, D = q.shape
    if page_table is None:
        Hkv, Lkv = k.shape[1], k.shape[2]
    else:
        Hkv, Lkv = k.shape[1], int(max_seq_len)
    a = PrefillArgs()
    if page_table is not None:
        a.page_table = page_table.data_ptr()
        a.seq_lens = seq_lens.data_ptr()
        a.num_pages, a.page_size = k.shape[0], k.shape[2]
        a.max_pages = page_table.shape[1]
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    a.out = out.data_ptr() if out is not None else None
    a.lse = lse.data_ptr() if lse is not None else None
    a.B, a.Hq, a.Hkv, a.Lq, a.Lkv, a.D = B, Hq, Hkv, Lq, Lkv, D
    a.causal = int(bool(causal))
    a.scale = float(scale if scale is not None else 1.0 / math.sqrt(D))
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    a.dtype = _DT[q.dtype]
    if mask is not None:
        m = mask if mask.dim() == 3 else mask.unsqueeze(0)
        a.mask = m.data_ptr()
        a.mask_dtype = _DT[m.dtype]
        a.mask_batches = m.shape[0]
    a.num_splits = int(num_splits)
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def fa_prefill_ex(q, k, v, *, causal=False, scale=None, mask=None, num_splits=0, out=None,
                  lse=None, workspace=None, stream=None):
    """Dense attention, any supported dtype (bf16/fp16/fp32), optional additive mask
    [1 or B, Lq, Lkv], optional KV split (0 = library's choice)."""
    lib = load_library()
    _need_dtype(q.dtype, k, v, out)
    _need_dtype(torch.float32, lse)
    _need_cuda(q, k, v, mask, out, lse)
    B, Hq, Lq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, Lq, dtype=torch.float32, device=q.device)
    a = prefill_args(q, k, v, causal=causal, scale=scale, out=out, lse=lse, mask=mask,
                     num_splits=num_splits)
    need = lib.fa_prefill_workspace_size(ctypes.byref(a))
    ws = _workspace(need, q.device, workspace)
    if ws is not None:
        a.workspace = ws.data_ptr()
        a.workspace_bytes = ws.numel() * ws.element_size()
    _check(lib.fa_prefill_ex(ctypes.byref(a), _stream(stream)))
    return out, lse


def prefill_workspace_size(q, k, v, **kw) -> int:
    return load_library().fa_prefill_workspace_size(ctypes.byref(prefill_args(q, k, v, **kw)))


def prefill_num_splits(q, k, v, **kw) -> int:
    return load_library().fa_prefill_num_splits(ctypes.byref(prefill_args(q, k, v, **kw)))


def fa_prefill_paged_workspace_size(B, Hq, Hkv, Lq, D, max_seq_len) -> int:
    return load_library().fa_prefill_paged_workspace_size(B, Hq, Hkv, Lq, D, max_seq_len)


def fa_prefill_paged(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int,
                     causal: bool = True, scale: float | None = None, mask=None, num_splits=0,
                     out=None, lse=None, workspace=None, stream=None):
    """Chunked prefill against a paged cache (fa_prefill_ex with a page table).
    q [B,Hq,Lq,D] bf16 or fp16 (each sequence's last Lq positions); pages
    [num_pages,Hkv,page_size,D] in q's dtype; page_table [B,max_pages] int32; seq_lens [B]
    int32 (device): each sequence's cached tokens, the chunk included; optional additive
    mask [1 or B, Lq, max_seq_len]."""
    lib = load_library()
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {q.dtype}")
    _need_dtype(q.dtype, k_pages, v_pages, out)
    _need_dtype(torch.int32, page_table, seq_lens)
    _need_dtype(torch.float32, lse)
    _need_cuda(q, k_pages, v_pages, page_table, seq_lens, mask, out, lse)
    B, Hq, Lq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, Lq, dtype=torch.float32, device=q.device)
    a = prefill_args(q, k_pages, v_pages, causal=causal, scale=scale, out=out, lse=lse,
                     mask=mask, num_splits=num_splits, page_table=page_table,
                     seq_lens=seq_lens, max_seq_len=max_seq_len)
    ws = _workspace(lib.fa_prefill_workspace_size(ctypes.byref(a)), q.device, workspace)
    if ws is not None:
        a.workspace = ws.data_ptr()
        a.workspace_bytes = ws.numel() * ws.element_size()
    _check(lib.fa_prefill_ex(ctypes.byref(a), _stream(stream)))
    return out, lse


def fa_decode_workspace_size(B, Hq, D, max_seq_len) -> int:
    return load_library().fa_decode_workspace_size(B, Hq, D, max_seq_len)


def decode_args(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int,
                scale: float | None = None, out=None, lse=None, workspace=None,
                path: int = FA_DECODE_AUTO) -> DecodeArgs:
    """Argument struct of fa_decode_paged_ex (sizes from the tensors' shapes)."""
    B, Hq, D = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {q.dtype}")
    return DecodeArgs(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(seq_lens),
                      _ptr(out), _ptr(lse), B, Hq, Hkv, D, page_size, page_table.shape[1],
                      num_pages, int(max_seq_len), float(scale), _DT[q.dtype], _ptr(workspace),
                      0 if workspace is None else workspace.numel() * workspace.element_size(),
                      int(path))


def fa_decode_get_plan(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int,
                       path: int = FA_DECODE_AUTO) -> dict:
    """What a decode call with these tensors does: {"path", "n_splits", "launches",
    "workspace_bytes"} (path 1 = CUDA cores, 2 = tensor cores)."""
    lib = load_library()
    a = decode_args(q, k_pages, v_pages, page_table, seq_lens, max_seq_len, path=path)
    pl = DecodePlan()
    _check(lib.fa_decode_get_plan(ctypes.byref(a), ctypes.byref(pl)))
    return {"path": pl.path, "n_splits": pl.n_splits, "launches": pl.launches,
            "workspace_bytes": pl.workspace_bytes}


def fa_decode_paged(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int,
                    scale: float | None = None, out=None, lse=None, workspace=None, stream=None,
                    path: int = FA_DECODE_AUTO):
    """Split-KV paged GQA decode.  q [B,Hq,D] bf16 or fp16; pages [num_pages,Hkv,page_size,D]
    in q's dtype; page_table [B,max_pages] int32; seq_lens [B] int32 (device).  path: 0 the
    library's choice, 1 the CUDA-core kernel, 2 the tensor-core kernel."""
    lib = load_library()
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {q.dtype}")
    _need_dtype(q.dtype, k_pages, v_pages)
    _need_dtype(torch.int32, page_table, seq_lens)
    _need_cuda(q, k_pages, v_pages, page_table, seq_lens)
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    _need_dtype(q.dtype, out)
    _need_dtype(torch.float32, lse)
    _need_cuda(out, lse)
    need = fa_decode_get_plan(q, k_pages, v_pages, page_table, seq_lens, max_seq_len,
                              path)["workspace_bytes"]
    ws = _workspace(need, q.device, workspace)
    a = decode_args(q, k_pages, v_pages, page_table, seq_lens, max_seq_len, scale, out, lse, ws,
                    path)
    _check(lib.fa_decode_paged_ex(ctypes.byref(a), _stream(stream)))
    return out, lse


def fa_decode_paged_noalloc(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int,
                            scale: float | None = None, out=None, lse=None, stream=None):
    """fa_decode_paged without a workspace, for callers that cannot allocate: the library's
    fixed device scratch is used instead (problems needing more than it holds are refused).
    Calls that overlap on the GPU share that scratch and race."""
    lib = load_library()
    _need_dtype(torch.bfloat16, q, k_pages, v_pages, out)
    _need_dtype(torch.int32, page_table, seq_lens)
    _need_dtype(torch.float32, lse)
    _need_cuda(q, k_pages, v_pages, page_table, seq_lens, out, lse)
    B, Hq, D = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    _check(lib.fa_decode_paged_noalloc(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                       _ptr(seq_lens), _ptr(out), _ptr(lse), B, Hq, Hkv, D,
                                       page_size, page_table.shape[1], num_pages,
                                       int(max_seq_len), float(scale), _stream(stream)))
    return out, lse


def fa_decode_chunk_tokens(B, Hq, max_seq_len) -> int:
    return load_library().fa_decode_chunk_tokens(B, Hq, max_seq_len)


def fa_decode_paged_states(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int,
                           scale: float | None = None, o_parts=None, lse_parts=None, stream=None):
    """Per-chunk split-KV states of paged decode (no merge).  Returns (o_parts
    [B*Hq, n_chunks, D] fp32, lse_parts [B*Hq, n_chunks] fp32, chunk)."""
    lib = load_library()
    _need_dtype(torch.bfloat16, q, k_pages, v_pages)
    _need_dtype(torch.int32, page_table, seq_lens)
    _need_cuda(q, k_pages, v_pages, page_table, seq_lens)
    B, Hq, D = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    chunk = lib.fa_decode_chunk_tokens(B, Hq, max_seq_len)
    n = -(-max_seq_len // chunk)
    if o_parts is None:
        o_parts = torch.empty(B * Hq, n, D, dtype=torch.float32, device=q.device)
    if lse_parts is None:
        lse_parts = torch.empty(B * Hq, n, dtype=torch.float32, device=q.device)
    _check(lib.fa_decode_paged_states(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                      _ptr(seq_lens), _ptr(o_parts), _ptr(lse_parts), n, B, Hq,
                                      Hkv, D, page_size, page_table.shape[1], num_pages,
                                      int(max_seq_len), float(scale), _stream(stream)))
    return o_parts, lse_parts, chunk


def mla_decode_chunk_tokens(B, H, max_seq_len) -> int:
    return load_library().mla_decode_chunk_tokens(B, H, max_seq_len)


def mla_decode_paged_states(q_nope, q_pe, ckv, kpe, page_table, seq_lens, max_seq_len: int,
                            scale: float, o_parts=None, lse_parts=None, stream=None):
    """Per-chunk split-KV states of MLA decode (no merge).  Returns (o_parts, lse_parts,
    chunk)."""
    lib = load_library()
    _need_dtype(torch.bfloat16, q_nope, q_pe, ckv, kpe)
    _need_dtype(torch.int32, page_table, seq_lens)
    _need_cuda(q_nope, q_pe, ckv, kpe, page_table, seq_lens)
    B, H, Dc = q_nope.shape
    Dr = q_pe.shape[2]
    num_pages, page_size = ckv.shape[0], ckv.shape[1]
    chunk = lib.mla_decode_chunk_tokens(B, H, max_seq_len)
    n = -(-max_seq_len // chunk)
    if o_parts is None:
        o_parts = torch.empty(B * H, n, Dc, dtype=torch.float32, device=q_nope.device)
    if lse_parts is None:
        lse_parts = torch.empty(B * H, n, dtype=torch.float32, device=q_nope.device)
    _check(lib.mla_decode_paged_states(_ptr(q_nope), _ptr(q_pe), _ptr(ckv), _ptr(kpe),
                                       _ptr(page_table), _ptr(seq_lens), _ptr(o_parts),
                                       _ptr(lse_parts), n, B, H, Dc, Dr, page_size,
                                       page_table.shape[1], num_pages, int(max_seq_len),
                                       float(scale), _stream(stream)))
    return o_parts, lse_parts, chunk


def mla_decode_workspace_size(B, H, Dc, max_seq_len) -> int:
    return load_library().mla_decode_workspace_size(B, H, Dc, max_seq_len)


def mla_decode_paged(q_nope, q_pe, ckv, kpe, page_table, seq_lens, max_seq_len: int,
                     scale: float, out=None, lse=None, workspace=None, stream=None):
    """MLA paged decode (latent form).  q_nope [B,H,512], q_pe [B,H,64] bf16 or fp16;
    ckv [P,page_size,512], kpe [P,page_size,64] in that dtype; page_table [B,max_pages];
    seq_lens [B]."""
    lib = load_library()
    if q_nope.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {q_nope.dtype}")
    _need_dtype(q_nope.dtype, q_pe, ckv, kpe)
    _need_dtype(torch.int32, page_table, seq_lens)
    _need_cuda(q_nope, q_pe, ckv, kpe, page_table, seq_lens)
    B, H, Dc = q_nope.shape
    Dr = q_pe.shape[2]
    num_pages, page_size = ckv.shape[0], ckv.shape[1]
    if out is None:
        out = torch.empty_like(q_nope)
    if lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=q_nope.device)
    _need_dtype(q_nope.dtype, out)
    _need_dtype(torch.float32, lse)
    _need_cuda(out, lse)
    ws = _workspace(lib.mla_decode_workspace_size(B, H, Dc, max_seq_len), q_nope.device, workspace)
    a = MlaArgs(_ptr(q_nope), _ptr(q_pe), _ptr(ckv), _ptr(kpe), _ptr(page_table), _ptr(seq_lens),
                _ptr(out), _ptr(lse), B, H, Dc, Dr, page_size, page_table.shape[1], num_pages,
                int(max_seq_len), float(scale), _DT[q_nope.dtype], _ptr(ws),
                0 if ws is None else ws.numel())
    _check(lib.mla_decode_paged_ex(ctypes.byref(a), _stream(stream)))
    return out, lse


def fa_merge_states(o_parts, lse_parts, n_splits=None, out_dtype=torch.bfloat16, out=None,
                    lse=None, stream=None):
    """Merge partial states: o_parts [rows,S,D] fp32, lse_parts [rows,S] fp32."""
    lib = load_library()
    _need_dtype(torch.float32, o_parts, lse_parts, lse)
    _need_dtype(torch.int32, n_splits)
    _need_cuda(o_parts, lse_parts, n_splits, out, lse)
    rows, S, D = o_parts.shape
    if out is None:
        out = torch.empty(rows, D, dtype=out_dtype, device=o_parts.device)
    if lse is None:
        lse = torch.empty(rows, dtype=torch.float32, device=o_parts.device)
    _check(lib.fa_merge_states(_ptr(o_parts), _ptr(lse_parts), _ptr(n_splits), _ptr(out),
                               _ptr(lse), rows, D, S, _DT[out.dtype], _stream(stream)))
    return out, lse


def fa_get_device_status(stream=None) -> int:
    """Synchronise, return and clear the library's sticky device status (0 = OK)."""
    return load_library().fa_get_device_status(_stream(stream))


def fa_selftest_wait_timeout(timeout_us: int, stream=None) -> int:
    """Enqueue the failure-path self-test (a bounded wait that runs out); returns the call's
    status.  Read the result with fa_get_device_status(): FA_ERR_TIMEOUT."""
    return load_library().fa_selftest_wait_timeout(int(timeout_us), _stream(stream))


def fa_last_error() -> str:
    return load_library().fa_last_error().decode(errors="replace")


def gated_delta_args(q, k, v, g, beta, *, scale=None, initial_state=None, out=None,
                     final_state=None, workspace=None) -> GatedDeltaArgs:
    """Argument struct of gated_delta_prefill (sizes from the tensors' shapes)."""
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    return GatedDeltaArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                          _ptr(out), _ptr(final_state), B, T, Hk, Hv, dk, dv, float(scale),
                          _DT[q.dtype], _ptr(workspace),
                          0 if workspace is None else workspace.numel() * workspace.element_size())


def gated_delta_workspace_size(q, k, v, g, beta) -> int:
    return load_library().gated_delta_workspace_size(
        ctypes.byref(gated_delta_args(q, k, v, g, beta)))


def gated_delta_prefill(q, k, v, g, beta, *, scale=None, initial_state=None, out=None,
                        final_state=None, want_state=True, workspace=None, stream=None):
    """Chunked prefill of gated-delta linear attention.  q, k [B,Hk,T,dk] bf16; v [B,Hv,T,dv]
    bf16; g (log decay), beta [B,Hv,T] fp32; initial_state [B,Hv,dv,dk] fp32 or None.
    Returns (out [B,Hv,T,dv] bf16, final state [B,Hv,dv,dk] fp32 or None)."""
    lib = load_library()
    _need_dtype(torch.bfloat16, q, k, v, out)
    _need_dtype(torch.float32, g, beta, initial_state, final_state)
    _need_cuda(q, k, v, g, beta, initial_state, out, final_state)
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    if out is None:
        out = torch.empty(B, Hv, T, dv, dtype=torch.bfloat16, device=q.device)
    if final_state is None and want_state:
        final_state = torch.empty(B, Hv, dv, dk, dtype=torch.float32, device=q.device)
    a = gated_delta_args(q, k, v, g, beta, scale=scale, initial_state=initial_state, out=out,
                         final_state=final_state)
    ws = _workspace(lib.gated_delta_workspace_size(ctypes.byref(a)), q.device, workspace)
    if ws is not None:
        a.workspace = ws.data_ptr()
        a.workspace_bytes = ws.numel() * ws.element_size()
    _check(lib.gated_delta_prefill(ctypes.byref(a), _stream(stream)))
    return out, final_state


# ------------------------------------------------------------------------------------------
# The serving step around the paged cache.  These calls take strided inputs, run on the
# tensors' own device whichever device is current, and allocate what they return (and any
# workspace) on the stream they launch on.
# ------------------------------------------------------------------------------------------
_CACHE_DT = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16, torch.float8_e4m3fn: FA_E4M3}
_STRUCT_CODE = {ctypes.c_void_p: "P", ctypes.c_int: "i", ctypes.c_float: "f", ctypes.c_size_t: "N",
                _Strides: "3q", _Strides2: "2q"}


def _packer(cls):
    """pack() of a structure's fields in order (arrays flattened): about a third of the time of
    filling a ctypes structure, which a decode step of a few microseconds feels."""
    st = struct.Struct("@" + "".join(_STRUCT_CODE[t] for _, t in cls._fields_))
    assert st.size <= ctypes.sizeof(cls) < st.size + 8  # C pads the end, struct does not
    pad = bytes(ctypes.sizeof(cls) - st.size)
    return (lambda *a: st.pack(*a) + pad) if pad else st.pack


_pack_rotary, _pack_append, _pack_gather, _pack_tree = map(
    _packer, (RotaryArgs, CacheAppendArgs, CacheGatherArgs, TreeArgs))
_pack_norm, _pack_norm_backward, _pack_packed, _pack_packed_backward, _pack_step = map(
    _packer, (NormRotaryArgs, NormRotaryBackwardArgs, PackedArgs, PackedBackwardArgs,
              GatedDeltaStepArgs))
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _Scope:
    """The device of a call's tensors and the stream it launches on, made current."""

    def __init__(self, dev, stream):
        self.device = torch.cuda.device(dev)
        self.stream = torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


_here = contextlib.nullcontext()


def _scope(dev, stream):
    if stream is None:
        return _here if dev == torch.cuda.current_device() else torch.cuda.device(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    return _Scope(dev, stream)


def _cuda_index(t):
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return t.get_device()


def _on(dev, *ts):
    """Contiguous tensors on device `dev` (None passes)."""
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors on one device")


def _strides_on(dev, t):
    """(batch, head, token) strides of a 4-D tensor on `dev` with a contiguous last dimension; 0
    for a dimension of one element, where torch may report anything."""
    s, n = t.stride(), t.shape
    if t.get_device() != dev or (s[3] != 1 and n[3] > 1):
        raise ValueError("tensors must be CUDA tensors on one device with a contiguous last "
                         "dimension")
    return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)


def _shape(name, t, *want):
    if t is not None and t.shape != want:
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")


def _addr(t):
    return 0 if t is None else t.data_ptr()


_ROTARY_SCALING = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}  # fa_rotary_scaling


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain",
                       factor: float = 1.0, original_len: float = 0.0, fast: float = 32.0,
                       slow: float = 1.0, device=None):
    """Table and amplitude of fa_rotary (and of fa_cache_append's rotation): (inv_freq [rot_dim/2]
    fp64 on `device`, amplitude).  scaling: "plain", "linear" (positions interpolated), "base" (the
    base raised), "by_parts" (YaRN; original_len is the training length)."""
    if scaling not in _ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY_SCALING)}, got {scaling!r}")
    table = torch.empty(max(rot_dim // 2, 0), dtype=torch.float64)
    amplitude = ctypes.c_float()
    lib = load_library()
    _check(lib.fa_rotary_frequencies(rot_dim, base, _ROTARY_SCALING[scaling], factor, original_len,
                                     fast, slow, table.data_ptr() or None, ctypes.byref(amplitude)))
    return (table if device is None else table.to(device)), amplitude.value


def tree_mask(parents, device=None):
    """fa_tree_decode_paged's mask of trees given by parents: [T] or [B,T] ints, parents[i] < i the
    drafted token before token i, -1 the context.  Returns int64 [1 or B,T,ceil(T/64)]."""
    p = torch.as_tensor(parents, dtype=torch.int32, device="cpu")
    p = (p if p.dim() == 2 else p.unsqueeze(0)).contiguous()
    B, T = p.shape
    words = torch.empty(B, T, -(-T // 64), dtype=torch.int64)
    lib = load_library()
    for b in range(B):
        _check(lib.fa_tree_mask(p[b].data_ptr(), T, words[b].data_ptr()))
    return words if device is None else words.to(device)


def fa_rotary(q, k, positions, inv_freq, *, amplitude: float = 1.0, interleaved: bool = False,
              transpose: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions on q [B,Hq,T,D] and k [B,Hk,T,D] (k may be None), bf16, fp16 or fp32,
    any strides with a contiguous last dimension; positions [B,T] int32; inv_freq [rot_dim/2]
    fp64: the first rot_dim columns of each head are rotated, in the half layout or interleaved,
    the rest copied.  transpose=True applies the transposed map, the gradient of the call.  q_out
    and k_out may be q and k themselves.  Returns (q_out, k_out)."""
    lib = load_library()
    dev = _cuda_index(q)
    B, Hq, T, D = q.shape
    Hk = 0 if k is None else k.shape[1]
    _need_dtype(q.dtype, k, q_out, k_out)
    _need_dtype(torch.int32, positions)
    _need_dtype(torch.float64, inv_freq)
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    _shape("k", k, B, Hk, T, D)
    _shape("q_out", q_out, B, Hq, T, D)
    _shape("k_out", k_out, B, Hk, T, D)
    _shape("positions", positions, B, T)
    _on(dev, positions, inv_freq)
    none = (0, 0, 0)
    with _scope(dev, stream):
        if q_out is None:
            q_out = torch.empty((B, Hq, T, D), dtype=q.dtype, device=q.device)
        if k is None:
            k_out = None
        elif k_out is None:
            k_out = torch.empty((B, Hk, T, D), dtype=q.dtype, device=q.device)
        a = _pack_rotary(q.data_ptr(), _addr(k), q_out.data_ptr(), _addr(k_out),
                         *_strides_on(dev, q), *(none if k is None else _strides_on(dev, k)),
                         *_strides_on(dev, q_out), *(none if k is None else _strides_on(dev, k_out)),
                         positions.data_ptr(), inv_freq.data_ptr(), B, T, Hq, Hk, D,
                         2 * inv_freq.numel(), interleaved, transpose, amplitude, _DT[q.dtype])
        _check(lib.fa_rotary(a, _raw_stream(dev)))
    return q_out, k_out


def _check_cache(dev, k_pages, v_pages, k_scales, v_scales, page_table, B):
    """(num_pages, Hkv, page_size, D) of a paged cache, its tensors checked."""
    dtype, shape = k_pages.dtype, k_pages.shape
    if dtype not in _CACHE_DT:
        raise ValueError(f"pages must be bfloat16, float16 or float8_e4m3fn, got {dtype}")
    _need_dtype(dtype, v_pages)
    _need_dtype(torch.int32, page_table)
    if len(shape) != 4:
        raise ValueError(f"pages must be [num_pages, Hkv, page_size, D], got {tuple(shape)}")
    _shape("v_pages", v_pages, *shape)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be [{B}, max_pages], got {tuple(page_table.shape)}")
    if dtype == torch.float8_e4m3fn:
        if k_scales is None or v_scales is None:
            raise ValueError("an 8-bit cache needs k_scales and v_scales")
        _need_dtype(torch.uint8, k_scales, v_scales)
        _shape("k_scales", k_scales, *shape[:3])
        _shape("v_scales", v_scales, *shape[:3])
    elif k_scales is not None or v_scales is not None:
        raise ValueError("scales belong to an 8-bit cache")
    _on(dev, k_pages, v_pages, k_scales, v_scales, page_table)
    return shape


def fa_cache_append(k, v, k_pages, v_pages, page_table, seq_lens, *, new_lens=None, k_scales=None,
                    v_scales=None, inv_freq=None, amplitude: float = 1.0,
                    interleaved: bool = False, positions=None, stream=None) -> None:
    """Write a step's k, v [B,Hkv,T,D] (any strides with a contiguous last dimension) into the
    pages [num_pages,Hkv,page_size,D]: in k's 16-bit type, or quantised (float8_e4m3fn pages,
    k_scales and v_scales [num_pages,Hkv,page_size] uint8).  seq_lens [B] int32 (device) counts
    the new tokens; sequence b has new_lens[b] of them (default T), its first rows.  With inv_freq
    [rot_dim/2] fp64 the keys are rotated on the way, at positions [B,T] int32 (default: the
    position in the cache)."""
    lib = load_library()
    dev = _cuda_index(k)
    B, Hkv, T, D = k.shape
    if k.dtype not in _DT:
        raise TypeError(f"unsupported dtype {k.dtype}")
    _need_dtype(k.dtype, v)
    _need_dtype(torch.int32, seq_lens, new_lens, positions)
    _need_dtype(torch.float64, inv_freq)
    _shape("v", v, B, Hkv, T, D)
    _shape("seq_lens", seq_lens, B)
    _shape("new_lens", new_lens, B)
    _shape("positions", positions, B, T)
    P, _, ps, _ = _check_cache(dev, k_pages, v_pages, k_scales, v_scales, page_table, B)
    _shape("k_pages", k_pages, P, Hkv, ps, D)
    _on(dev, seq_lens, new_lens, positions, inv_freq)
    a = _pack_append(k.data_ptr(), v.data_ptr(), *_strides_on(dev, k), *_strides_on(dev, v),
                     k_pages.data_ptr(), v_pages.data_ptr(), _addr(k_scales), _addr(v_scales),
                     page_table.data_ptr(), seq_lens.data_ptr(), _addr(new_lens), _addr(positions),
                     _addr(inv_freq), B, T, Hkv, D, ps, page_table.shape[1], P,
                     0 if inv_freq is None else 2 * inv_freq.numel(), interleaved, amplitude,
                     _DT[k.dtype], _CACHE_DT[k_pages.dtype])
    with _scope(dev, stream):
        _check(lib.fa_cache_append(a, _raw_stream(dev)))


def fa_cache_gather(k_pages, v_pages, page_table, seq_lens, max_seq_len: int, *,
                    dtype=torch.bfloat16, k_scales=None, v_scales=None, k=None, v=None,
                    stream=None):
    """Read a paged cache (bf16, fp16, or float8_e4m3fn with its scales) back as dense k, v
    [B,Hkv,max_seq_len,D] in dtype; rows at and past seq_lens[b] are zero."""
    lib = load_library()
    dev = _cuda_index(k_pages)
    B, L = seq_lens.shape[0], int(max_seq_len)
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    _need_dtype(dtype, k, v)
    _need_dtype(torch.int32, seq_lens)
    _shape("seq_lens", seq_lens, B)
    P, Hkv, ps, D = _check_cache(dev, k_pages, v_pages, k_scales, v_scales, page_table, B)
    _shape("k", k, B, Hkv, L, D)
    _shape("v", v, B, Hkv, L, D)
    _on(dev, seq_lens, k, v)
    with _scope(dev, stream):
        if k is None:
            k = torch.empty((B, Hkv, L, D), dtype=dtype, device=k_pages.device)
        if v is None:
            v = torch.empty((B, Hkv, L, D), dtype=dtype, device=k_pages.device)
        a = _pack_gather(k_pages.data_ptr(), v_pages.data_ptr(), _addr(k_scales), _addr(v_scales),
                         page_table.data_ptr(), seq_lens.data_ptr(), k.data_ptr(), v.data_ptr(), B,
                         Hkv, D, ps, page_table.shape[1], P, L, _DT[dtype],
                         _CACHE_DT[k_pages.dtype])
        _check(lib.fa_cache_gather(a, _raw_stream(dev)))
    return k, v


def fa_tree_decode_paged(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: int, *,
                         tree_mask=None, draft_lens=None, scale: float | None = None,
                         k_scales=None, v_scales=None, num_splits: int = 0, out=None, lse=None,
                         workspace=None, stream=None):
    """Attention of a tree of drafted tokens, each sequence's last draft_lens[b] (default T)
    tokens in the cache.  q [B,Hq,T,D] bf16 or fp16 (any strides with a contiguous last
    dimension); pages [num_pages,Hkv,page_size,D] in q's dtype, or float8_e4m3fn with k_scales
    and v_scales [num_pages,Hkv,page_size] uint8; seq_lens [B] int32 (device) counts the drafted
    tokens; tree_mask [1 or B,T,ceil(T/64)] int64: bit j of row i = query i sees drafted token j
    (None: a chain).  T = 1 is the decode of one token a sequence.  Returns (out [B,Hq,T,D], lse
    [B,Hq,T] fp32)."""
    lib = load_library()
    dev = _cuda_index(q)
    B, Hq, T, D = q.shape
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {q.dtype}")
    _need_dtype(q.dtype, out)
    _need_dtype(torch.float32, lse)
    _need_dtype(torch.int32, seq_lens, draft_lens)
    _need_dtype(torch.int64, tree_mask)
    _shape("seq_lens", seq_lens, B)
    _shape("draft_lens", draft_lens, B)
    _shape("out", out, B, Hq, T, D)
    _shape("lse", lse, B, Hq, T)
    P, Hkv, ps, Dk = _check_cache(dev, k_pages, v_pages, k_scales, v_scales, page_table, B)
    if Dk != D or (k_scales is None and k_pages.dtype != q.dtype):
        raise ValueError(f"pages of {Dk} columns in {k_pages.dtype} do not go with q's {D} in {q.dtype}")
    masks = 0
    if tree_mask is not None:
        masks = tree_mask.shape[0]
        if masks not in (1, B) or tree_mask.shape[1:] != (T, -(-T // 64)):
            raise ValueError(f"tree_mask must be [1 or {B}, {T}, {-(-T // 64)}], got {tuple(tree_mask.shape)}")
    _on(dev, seq_lens, draft_lens, tree_mask, out, lse, workspace)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((B, Hq, T, D), dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
        fields = (q.data_ptr(), *_strides_on(dev, q), k_pages.data_ptr(), v_pages.data_ptr(),
                  _addr(k_scales), _addr(v_scales), page_table.data_ptr(), seq_lens.data_ptr(),
                  _addr(draft_lens), _addr(tree_mask), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv,
                  T, D, ps, page_table.shape[1], P, int(max_seq_len), masks, int(num_splits),
                  1.0 / math.sqrt(D) if scale is None else scale, _DT[q.dtype],
                  _CACHE_DT[k_pages.dtype])
        a = _pack_tree(*fields, 0, 0)
        need = lib.fa_tree_workspace_size(a)
        if need:
            ws = _workspace(need, q.device, workspace)
            a = _pack_tree(*fields, ws.data_ptr(), ws.numel() * ws.element_size())
        _check(lib.fa_tree_decode_paged(a, _raw_stream(dev)))
    return out, lse


# ------------------------------------------------------------------------------------------
# Packed prompts, forward and backward; norms of queries and keys; the recurrent gated-delta step.
# As above: strided inputs, the tensors' own device, allocations on the launching stream.  A call of
# these on a few tokens takes the GPU about as long as Python takes to look at its arguments, so each
# tensor is looked at once, and what is wrong is found out only where something is.
# ------------------------------------------------------------------------------------------
_HALF = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}
_none3 = (0, 0, 0)
_empty = torch.empty


def _gpu(t):
    """Device index of a CUDA tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    return dev


def _flat(dev, dtype, shape, name, t):
    """Address of a contiguous tensor of this type and shape on the device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _need_dtype(dtype, t)
        _shape(name, t, *shape)
        _on(dev, t)
    return t.data_ptr()


def _strided(dev, dtype, shape, name, t):
    """Strides but the last of a tensor of this type and shape (three or four dimensions) on the
    device, contiguous in its last dimension; 0 for a dimension of one element, where torch may
    report anything."""
    s = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or (s[-1] != 1 and shape[-1] > 1):
        _need_dtype(dtype, t)
        _shape(name, t, *shape)
        raise ValueError("tensors must be CUDA tensors on one device with a contiguous last "
                         "dimension")
    if len(s) == 3:
        return (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0)
    return (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)


def _norm_fields(dev, shape, Hk, dtype, positions, inv_freq, q_weight, k_weight, amplitude,
                 interleaved, eps):
    """The checked fields that fa_qk_norm_rotary and its backward share."""
    B, Hq, T, D = shape
    code = _DT.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    wq = wk = pos = freq = rot = 0
    wcode = code
    weight = k_weight if q_weight is None else q_weight
    if weight is not None:
        wtype = weight.dtype
        wcode = _DT.get(wtype)
        if wtype is not dtype and wtype is not torch.float32:
            raise ValueError(f"the weights must be {dtype} or float32, got {wtype}")
        if q_weight is not None:
            wq = _flat(dev, wtype, (D,), "q_weight", q_weight)
        if k_weight is not None:
            wk = _flat(dev, wtype, (D,), "k_weight", k_weight)
    if positions is not None and inv_freq is not None:
        pos = _flat(dev, torch.int32, (B, T), "positions", positions)
        freq = _flat(dev, torch.float64, inv_freq.shape, "inv_freq", inv_freq)
        rot = 2 * inv_freq.numel()
    elif positions is not None or inv_freq is not None:
        raise ValueError("positions and inv_freq go together")
    return wq, wk, pos, freq, B, T, Hq, Hk, D, rot, interleaved, amplitude, eps, code, wcode


def fa_qk_norm_rotary(q, k, positions, inv_freq, q_weight, k_weight=None, *, eps: float = 1e-6,
                      amplitude: float = 1.0, interleaved: bool = False, q_out=None, k_out=None,
                      stream=None):
    """RMS norms of q [B,Hq,T,D] and k [B,Hk,T,D] (k may be None) for each head, times q_weight and
    k_weight [D] (q's dtype or fp32; None: ones), then fa_rotary's rotation, in one pass.  bf16,
    fp16 or fp32, any strides with a contiguous last dimension; positions [B,T] int32 and inv_freq
    [rot_dim/2] fp64, or None for both: norms alone.  q_out and k_out may be q and k themselves.
    Returns (q_out, k_out)."""
    lib = _lib or load_library()
    dev, dtype, qs = _gpu(q), q.dtype, q.shape
    B, _, T, D = qs
    q_in = _strided(dev, dtype, qs, "q", q)
    ka, Hk, k_in, k_to = 0, 0, _none3, _none3
    if k is not None:
        Hk = k.shape[1]
        ks = (B, Hk, T, D)
        ka, k_in = k.data_ptr(), _strided(dev, dtype, ks, "k", k)
    fields = _norm_fields(dev, qs, Hk, dtype, positions, inv_freq, q_weight, k_weight, amplitude,
                          interleaved, eps)
    with _scope(dev, stream):
        if q_out is None:
            q_out = _empty(qs, dtype=dtype, device=q.device)
        if k is None:
            k_out = None
        else:
            if k_out is None:
                k_out = _empty(ks, dtype=dtype, device=q.device)
            k_to = _strided(dev, dtype, ks, "k_out", k_out)
        a = _pack_norm(q.data_ptr(), ka, q_out.data_ptr(), 0 if k is None else k_out.data_ptr(), *q_in,
                       *k_in, *_strided(dev, dtype, qs, "q_out", q_out), *k_to, *fields)
        _check(lib.fa_qk_norm_rotary(a, _raw_stream(dev)))
    return q_out, k_out


def fa_qk_norm_rotary_backward(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight=None, *,
                               eps: float = 1e-6, amplitude: float = 1.0, interleaved: bool = False,
                               dq=None, dk=None, workspace=None, stream=None):
    """Gradient of fa_qk_norm_rotary: of the outputs' gradients dq_out, dk_out and the call's
    inputs.  dq and dk may be dq_out and dk_out, or q and k, themselves.  Returns (dq, dk, dq_weight,
    dk_weight): the last two [D] fp32, None where there is no weight."""
    lib = _lib or load_library()
    dev, dtype, qs = _gpu(q), q.dtype, q.shape
    B, _, T, D = qs
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    q_in = _strided(dev, dtype, qs, "q", q)
    q_back = _strided(dev, dtype, qs, "dq_out", dq_out)
    ka, ga, Hk, k_in, k_back, k_to = 0, 0, 0, _none3, _none3, _none3
    if k is not None:
        Hk = k.shape[1]
        ks = (B, Hk, T, D)
        ka, k_in = k.data_ptr(), _strided(dev, dtype, ks, "k", k)
        ga, k_back = dk_out.data_ptr(), _strided(dev, dtype, ks, "dk_out", dk_out)
    fields = _norm_fields(dev, qs, Hk, dtype, positions, inv_freq, q_weight, k_weight, amplitude,
                          interleaved, eps)
    if workspace is not None:
        _on(dev, workspace)
    device = q.device
    with _scope(dev, stream):
        if dq is None:
            dq = _empty(qs, dtype=dtype, device=device)
        if k is None:
            dk = None
        else:
            if dk is None:
                dk = _empty(ks, dtype=dtype, device=device)
            k_to = _strided(dev, dtype, ks, "dk", dk)
        dqw = None if q_weight is None else _empty((D,), dtype=torch.float32, device=device)
        dkw = None if k_weight is None else _empty((D,), dtype=torch.float32, device=device)
        fields = (dq_out.data_ptr(), ga, q.data_ptr(), ka, dq.data_ptr(), _addr(dk), _addr(dqw),
                  _addr(dkw), *q_back, *k_back, *q_in, *k_in, *_strided(dev, dtype, qs, "dq", dq),
                  *k_to, *fields)
        need = lib.fa_qk_norm_rotary_backward_workspace_size(_pack_norm_backward(*fields, 0, 0))
        ws = _workspace(need, device, workspace)
        a = _pack_norm_backward(*fields, _addr(ws), 0 if ws is None else ws.numel() * ws.element_size())
        _check(lib.fa_qk_norm_rotary_backward(a, _raw_stream(dev)))
    return dq, dk, dqw, dkw


def _packed_fields(dev, dtype, q, k, cu_seqlens_q, cu_seqlens_k, causal, scale):
    """The checked fields that fa_prefill_packed and its backward share."""
    code = _HALF.get(dtype)
    if code is None:
        raise ValueError(f"expected bfloat16 or float16, got {dtype}")
    if len(q) != 3 or len(k) != 3:
        raise ValueError("q, k and v must be [tokens, heads, D]")
    total_q, Hq, D = q
    total_k, Hkv, _ = k
    n = cu_seqlens_q.shape
    if len(n) != 1 or n[0] < 1:
        raise ValueError("cu_seqlens_q must be [B + 1]")
    at_q = at_k = _flat(dev, torch.int32, n, "cu_seqlens_q", cu_seqlens_q)
    if cu_seqlens_k is not None:
        at_k = _flat(dev, torch.int32, n, "cu_seqlens_k", cu_seqlens_k)
    elif total_k != total_q:
        raise ValueError("without cu_seqlens_k the keys are the queries' tokens: "
                         f"got {total_q} rows of q and {total_k} of k")
    return (at_q, at_k, n[0] - 1, Hq, Hkv, D, total_q, total_k, causal,
            1.0 / math.sqrt(D) if scale is None else scale, code)


def fa_prefill_packed(q, k, v, cu_seqlens_q, cu_seqlens_k=None, *, causal: bool = True,
                      scale: float | None = None, num_splits: int = 0, out=None, lse=None,
                      workspace=None, stream=None):
    """Attention over packed prompts: q [total_q,Hq,D], k, v [total_k,Hkv,D] bf16 or fp16 (any
    token and head strides with a contiguous last dimension, as slices of one projection), the
    sequences behind one another; cu_seqlens_q, cu_seqlens_k [B+1] int32 (device): first row of
    each and the end of the last (cu_seqlens_k None: the same).  causal: a sequence's queries are
    its last positions.  num_splits: parts of each sequence's keys (0: the library's choice).  Rows
    outside the sequences are left as they were.  Returns (out [total_q,Hq,D], lse [total_q,Hq]
    fp32)."""
    lib = _lib or load_library()
    dev, dtype, qs, ks = _gpu(q), q.dtype, q.shape, k.shape
    fields = _packed_fields(dev, dtype, qs, ks, cu_seqlens_q, cu_seqlens_k, causal, scale)
    rows = qs[:2]
    ks = (ks[0], ks[1], qs[2])
    strides = (*_strided(dev, dtype, qs, "q", q), *_strided(dev, dtype, ks, "k", k),
               *_strided(dev, dtype, ks, "v", v))
    with _scope(dev, stream):
        if out is None:
            out = _empty(qs, dtype=dtype, device=q.device)
        if lse is None:
            lse = _empty(rows, dtype=torch.float32, device=q.device)
        fields = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                  _flat(dev, torch.float32, rows, "lse", lse), *strides,
                  *_strided(dev, dtype, qs, "out", out), *fields, num_splits)
        a = _pack_packed(*fields, 0, 0)
        # (keys of fewer than 2048 a sequence are in parts only where the caller asks for it: twice the eight tiles of
        # 128 keys that a part of the library's own choice has at least)
        if num_splits > 1 or (num_splits == 0 and ks[0] >= 2048 * (len(cu_seqlens_q) - 1)):
            need = lib.fa_packed_workspace_size(a)
            if need:
                if workspace is not None:
                    _on(dev, workspace)
                ws = _workspace(need, q.device, workspace)
                a = _pack_packed(*fields, ws.data_ptr(), ws.numel() * ws.element_size())
        _check(lib.fa_prefill_packed(a, _raw_stream(dev)))
    return out, lse


def fa_prefill_packed_backward(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k=None, *,
                               causal: bool = True, scale: float | None = None, dq=None, dk=None,
                               dv=None, workspace=None, stream=None):
    """Gradients of fa_prefill_packed's out: dout [total_q,Hq,D], the call's inputs, and the out and
    lse that it returned.  Rows of dq, dk and dv outside the sequences are left as they were.
    Returns (dq [total_q,Hq,D], dk, dv [total_k,Hkv,D])."""
    lib = _lib or load_library()
    dev, dtype, qs, ks = _gpu(q), q.dtype, q.shape, k.shape
    fields = _packed_fields(dev, dtype, qs, ks, cu_seqlens_q, cu_seqlens_k, causal, scale)
    ks = (ks[0], ks[1], qs[2])
    strides = (*_strided(dev, dtype, qs, "dout", dout), *_strided(dev, dtype, qs, "q", q),
               *_strided(dev, dtype, ks, "k", k), *_strided(dev, dtype, ks, "v", v),
               *_strided(dev, dtype, qs, "out", out))
    at_lse = _flat(dev, torch.float32, qs[:2], "lse", lse)
    if workspace is not None:
        _on(dev, workspace)
    device = q.device
    with _scope(dev, stream):
        if dq is None:
            dq = _empty(qs, dtype=dtype, device=device)
        if dk is None:
            dk = _empty(ks, dtype=dtype, device=device)
        if dv is None:
            dv = _empty(ks, dtype=dtype, device=device)
        fields = (dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), at_lse,
                  dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *strides,
                  *_strided(dev, dtype, qs, "dq", dq), *_strided(dev, dtype, ks, "dk", dk),
                  *_strided(dev, dtype, ks, "dv", dv), *fields)
        need = lib.fa_packed_backward_workspace_size(_pack_packed_backward(*fields, 0, 0))
        ws = _workspace(need, device, workspace)
        a = _pack_packed_backward(*fields, _addr(ws), 0 if ws is None else ws.numel() * ws.element_size())
        _check(lib.fa_prefill_packed_backward(a, _raw_stream(dev)))
    return dq, dk, dv


def gated_delta_step(q, k, v, g, beta, states, *, read_index=None, write_index=None, new_lens=None,
                     scale: float | None = None, out=None, stream=None):
    """The gated delta rule over the next T tokens of each sequence, one after another: q, k
    [B,Hk,T,128], v [B,Hv,T,128] bf16 or fp16 (any strides with a contiguous last dimension); g
    (log decay), beta [B,Hv,T] fp32, any strides; states [num_states,Hv,128,128] fp32, updated.
    Sequence b's state is read from slot read_index[b] (default b) and written to write_index[b]
    (default where it was read); it has new_lens[b] tokens (default T; int32, device, all three).
    Returns out [B,Hv,T,128]."""
    lib = _lib or load_library()
    dev, dtype, qs = _gpu(q), q.dtype, q.shape
    code = _HALF.get(dtype)
    if code is None:
        raise ValueError(f"expected bfloat16 or float16, got {dtype}")
    B, Hk, T, dk = qs
    Hv, dv = v.shape[1], v.shape[3]
    vs, gate, n = (B, Hv, T, dv), (B, Hv, T), states.shape[0]
    for name, t in (("g", g), ("beta", beta)):
        if t.dtype is not torch.float32 or t.shape != gate or t.get_device() != dev:
            _need_dtype(torch.float32, t)
            _shape(name, t, *gate)
            raise ValueError("tensors must be CUDA tensors on one device")
    at_states = _flat(dev, torch.float32, (n, Hv, dv, dk), "states", states)
    i32 = torch.int32
    read = 0 if read_index is None else _flat(dev, i32, (B,), "read_index", read_index)
    write = 0 if write_index is None else _flat(dev, i32, (B,), "write_index", write_index)
    lens = 0 if new_lens is None else _flat(dev, i32, (B,), "new_lens", new_lens)
    strides = (*_strided(dev, dtype, qs, "q", q), *_strided(dev, dtype, qs, "k", k),
               *_strided(dev, dtype, vs, "v", v), *g.stride(), *beta.stride())
    with _scope(dev, stream):
        if out is None:
            out = _empty(vs, dtype=dtype, device=q.device)
        a = _pack_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                       at_states, read, write, lens, out.data_ptr(), *strides,
                       *_strided(dev, dtype, vs, "out", out), B, T, Hk, Hv, dk, dv, n,
                       1.0 / math.sqrt(dk) if scale is None else scale, code)
        _check(lib.gated_delta_step(a, _raw_stream(dev)))
    return out
