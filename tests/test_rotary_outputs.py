"""Host-side checks of fa_rotary's outputs: rows that would be written over one another are refused
before anything is enqueued, so no device is needed."""
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


def _args(q_out_s, k_out_s, **kw):
    st = ctypes.c_int64 * 3
    a = fa.RotaryArgs()
    for name, v in {**dict(q=P, k=P, q_out=P, k_out=P, q_strides=st(0, 0, 0), k_strides=st(0, 0, 0),
                           q_out_strides=st(*q_out_s), k_out_strides=st(*k_out_s), positions=P, inv_freq=P, B=2,
                           T=3, Hq=4, Hk=2, D=128, rot_dim=128, amplitude=1.0, dtype=fa.FA_BF16), **kw}.items():
        setattr(a, name, v)
    return a


GOOD = (1536, 128, 512)


@pytest.mark.parametrize("bad", [(0, 128, 512), (1536, 0, 512), (1536, 128, 0), (1536, 64, 512), (1536, 128, -64)])
@pytest.mark.parametrize("which", [0, 1])
def test_overlapping_rows_are_refused(lib, bad, which):
    a = _args(bad, GOOD) if which == 0 else _args(GOOD, bad)
    assert lib.fa_rotary(ctypes.byref(a), None) == fa.FA_ERR_INVALID_ARG
    assert "overlap" in fa.fa_last_error()


@pytest.mark.parametrize("kw,strides", [(dict(B=1), (0, 128, 512)), (dict(T=1), (1536, 128, 0)), (dict(Hq=1), (1536, 0, 512))])
def test_dimensions_of_one_need_no_stride(lib, kw, strides):
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are none")
    a = _args(strides, GOOD, **kw)
    assert lib.fa_rotary(ctypes.byref(a), None) == fa.FA_ERR_CUDA


def test_a_missing_side_is_not_looked_at(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are none")
    a = _args((0, 0, 0), GOOD, Hq=0, q=None, q_out=None)
    assert lib.fa_rotary(ctypes.byref(a), None) == fa.FA_ERR_CUDA
