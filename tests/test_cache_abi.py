"""Host-side refusals of the serving-step calls (rotary positions, cache write and read): every
bad argument is answered with its status code and a message before anything is enqueued, so no
device is needed."""
import ctypes

import pytest
import torch

import softmax_attention_gb300 as fa
from softmax_attention_gb300 import build as fa_build

P = 4096  # a non-null, aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def _fill(a, base, kw):
    for k, v in {**base, **kw}.items():
        if k.endswith("_strides"):
            v = (ctypes.c_int64 * 3)(*v)
        setattr(a, k, v)
    return a


def _rotary(**kw):
    s = (1024, 128, 512)
    return _fill(fa.RotaryArgs(), dict(
        q=P, k=P, q_out=P, k_out=P, q_strides=s, k_strides=s, q_out_strides=s, k_out_strides=s,
        positions=P, inv_freq=P, B=1, T=2, Hq=4, Hk=2, D=128, rot_dim=128, amplitude=1.0,
        dtype=fa.FA_BF16), kw)


def _append(**kw):
    s = (1024, 128, 512)
    return _fill(fa.CacheAppendArgs(), dict(
        k=P, v=P, k_strides=s, v_strides=s, k_pages=P, v_pages=P, k_scales=P, v_scales=P,
        page_table=P, seq_lens=P, B=1, T=2, Hkv=2, D=128, page_size=16, max_pages=4, num_pages=4,
        amplitude=1.0, dtype=fa.FA_BF16, cache_dtype=fa.FA_E4M3), kw)


def _gather(**kw):
    return _fill(fa.CacheGatherArgs(), dict(
        k_pages=P, v_pages=P, k_scales=P, v_scales=P, page_table=P, seq_lens=P, k=P, v=P, B=1,
        Hkv=2, D=128, page_size=16, max_pages=4, num_pages=4, max_seq_len=64, dtype=fa.FA_BF16,
        cache_dtype=fa.FA_E4M3), kw)


INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
CASES = [
    ("fa_rotary", _rotary, dict(B=-1), INV),
    ("fa_rotary", _rotary, dict(T=-1), INV),
    ("fa_rotary", _rotary, dict(D=0), INV),
    ("fa_rotary", _rotary, dict(D=100, rot_dim=64), UNS),
    ("fa_rotary", _rotary, dict(rot_dim=0), UNS),
    ("fa_rotary", _rotary, dict(rot_dim=24), UNS),
    ("fa_rotary", _rotary, dict(rot_dim=144), UNS),
    ("fa_rotary", _rotary, dict(D=1024, rot_dim=1024), UNS),
    ("fa_rotary", _rotary, dict(dtype=fa.FA_E4M3), UNS),
    ("fa_rotary", _rotary, dict(amplitude=float("nan")), INV),
    ("fa_rotary", _rotary, dict(q=P + 2), INV),
    ("fa_rotary", _rotary, dict(k_out=None), INV),
    ("fa_rotary", _rotary, dict(inv_freq=None), INV),
    ("fa_rotary", _rotary, dict(q_strides=(1024, 132, 512)), INV),
    ("fa_cache_append", _append, dict(T=-1), INV),
    ("fa_cache_append", _append, dict(D=96), UNS),
    ("fa_cache_append", _append, dict(page_size=24), INV),
    ("fa_cache_append", _append, dict(Hkv=0), INV),
    ("fa_cache_append", _append, dict(dtype=fa.FA_E4M3), UNS),
    ("fa_cache_append", _append, dict(cache_dtype=fa.FA_FP16), UNS),
    ("fa_cache_append", _append, dict(dtype=fa.FA_FP32, cache_dtype=fa.FA_FP32), UNS),
    ("fa_cache_append", _append, dict(k_scales=None), INV),
    ("fa_cache_append", _append, dict(inv_freq=P, rot_dim=256), UNS),
    ("fa_cache_append", _append, dict(inv_freq=P, rot_dim=64, amplitude=float("inf")), INV),
    ("fa_cache_append", _append, dict(page_table=None), INV),
    ("fa_cache_append", _append, dict(v=P + 8), INV),
    ("fa_cache_append", _append, dict(k_strides=(1024, 128, 4)), INV),
    ("fa_cache_append", _append, dict(max_pages=1 << 28), UNS),
    ("fa_cache_gather", _gather, dict(max_seq_len=65), INV),
    ("fa_cache_gather", _gather, dict(max_seq_len=-1), INV),
    ("fa_cache_gather", _gather, dict(cache_dtype=fa.FA_FP32), UNS),
    ("fa_cache_gather", _gather, dict(dtype=fa.FA_E4M3), UNS),
    ("fa_cache_gather", _gather, dict(v_scales=None), INV),
    ("fa_cache_gather", _gather, dict(D=32), UNS),
    ("fa_cache_gather", _gather, dict(k=None), INV),
    ("fa_cache_gather", _gather, dict(B=40000), UNS),
]


@pytest.mark.parametrize("name,make,kw,code", CASES)
def test_refusals(lib, name, make, kw, code):
    a = make(**kw)
    assert getattr(lib, name)(ctypes.byref(a), None) == code, lib.fa_last_error()
    assert name.encode() in lib.fa_last_error()


@pytest.mark.parametrize("name,make,kw", [
    ("fa_rotary", _rotary, dict(B=0)), ("fa_rotary", _rotary, dict(T=0)),
    ("fa_rotary", _rotary, dict(Hq=0, Hk=0)), ("fa_cache_append", _append, dict(T=0)),
    ("fa_cache_append", _append, dict(B=0)), ("fa_cache_gather", _gather, dict(max_seq_len=0)),
    ("fa_cache_gather", _gather, dict(B=0)),
])
def test_empty_work_needs_no_device(lib, name, make, kw):
    assert getattr(lib, name)(ctypes.byref(make(**kw)), None) == fa.FA_OK


@pytest.mark.parametrize("name", ["fa_rotary", "fa_cache_append", "fa_cache_gather"])
def test_null_struct(lib, name):
    assert getattr(lib, name)(None, None) == fa.FA_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_rotary(x, None, i, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        fa.fa_cache_append(x, x, x, x, i, i[0, :1])
    with pytest.raises(ValueError):
        fa.fa_cache_gather(x, x, i, i[0, :1], 3)
