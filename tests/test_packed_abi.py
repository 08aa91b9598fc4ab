"""Host-side checks of the packed-prompt calls, the norms with rotary positions and the recurrent
gated-delta step: every bad argument is answered with its status code and a message before anything
is enqueued, so no device is needed."""
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
            v = (ctypes.c_int64 * len(v))(*v)
        setattr(a, k, v)
    return a


def _packed(**kw):
    s = (1024, 128)
    return _fill(fa.PackedArgs(), dict(
        q=P, k=P, v=P, out=P, lse=P, q_strides=s, k_strides=s, v_strides=s, out_strides=s,
        cu_seqlens_q=P, cu_seqlens_k=P, B=2, Hq=4, Hkv=2, D=128, total_q=9, total_k=9, causal=1,
        scale=0.1, dtype=fa.FA_BF16), kw)


def _packed_backward(**kw):
    s = (1024, 128)
    names = ("dout", "q", "k", "v", "out", "dq", "dk", "dv")
    return _fill(fa.PackedBackwardArgs(), dict(
        {n: P for n in names}, **{n + "_strides": s for n in names}, lse=P, cu_seqlens_q=P,
        cu_seqlens_k=P, B=2, Hq=4, Hkv=2, D=128, total_q=9, total_k=9, causal=1, scale=0.1,
        dtype=fa.FA_BF16, workspace=P, workspace_bytes=1 << 20), kw)


def _norm(**kw):
    s = (1024, 128, 512)
    return _fill(fa.NormRotaryArgs(), dict(
        q=P, k=P, q_out=P, k_out=P, q_strides=s, k_strides=s, q_out_strides=s, k_out_strides=s,
        q_weight=P, k_weight=P, positions=P, inv_freq=P, B=1, T=2, Hq=4, Hk=2, D=128, rot_dim=128,
        amplitude=1.0, eps=1e-6, dtype=fa.FA_BF16, weight_dtype=fa.FA_BF16), kw)


def _norm_backward(**kw):
    s = (1024, 128, 512)
    names = ("dq_out", "dk_out", "q", "k", "dq", "dk")
    return _fill(fa.NormRotaryBackwardArgs(), dict(
        {n: P for n in names}, **{n + "_strides": s for n in names}, dq_weight=P, dk_weight=P,
        q_weight=P, k_weight=P, positions=P, inv_freq=P, B=1, T=2, Hq=4, Hk=2, D=128, rot_dim=128,
        amplitude=1.0, eps=1e-6, dtype=fa.FA_BF16, weight_dtype=fa.FA_FP32, workspace=P,
        workspace_bytes=1 << 24), kw)


def _step(**kw):
    s, g = (1024, 128, 512), (8, 2, 1)
    return _fill(fa.GatedDeltaStepArgs(), dict(
        q=P, k=P, v=P, g=P, beta=P, states=P, out=P, q_strides=s, k_strides=s, v_strides=s,
        g_strides=g, beta_strides=g, out_strides=s, B=1, T=2, Hk=2, Hv=4, dk=128, dv=128,
        num_states=1, scale=0.1, dtype=fa.FA_BF16), kw)


INV, UNS, WS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")
SIZES = [  # of the packed calls, both directions
    (dict(B=-1), INV), (dict(total_q=-1), INV), (dict(total_k=-2), INV), (dict(Hq=5), INV),
    (dict(Hkv=0), INV), (dict(Hq=258), UNS), (dict(D=96), UNS), (dict(D=256), UNS),
    (dict(dtype=fa.FA_FP32), UNS), (dict(dtype=fa.FA_E4M3), UNS), (dict(scale=NAN), INV),
    (dict(scale=INF), INV), (dict(cu_seqlens_q=None), INV), (dict(cu_seqlens_k=None), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=P + 2), INV), (dict(q_strides=(1024, 0)), INV),
    (dict(k_strides=(1028, 128)), INV), (dict(v_strides=(-1024, 128)), INV),
    (dict(k_strides=(64, 128)), INV), (dict(total_q=1 << 30, Hq=65536, Hkv=65536), UNS),
]
CASES = (
    [("fa_prefill_packed", _packed, kw, code) for kw, code in SIZES]
    + [("fa_prefill_packed", _packed, kw, code) for kw, code in [
        (dict(out=None), INV), (dict(out=P + 8), INV), (dict(out_strides=(0, 128)), INV)]]
    + [("fa_prefill_packed_backward", _packed_backward, kw, code) for kw, code in SIZES]
    + [("fa_prefill_packed_backward", _packed_backward, kw, code) for kw, code in [
        (dict(dout=None), INV), (dict(out=None), INV), (dict(lse=None), INV), (dict(lse=P + 2), INV),
        (dict(dq=None), INV), (dict(dk=P + 4), INV), (dict(dv_strides=(1024, 64)), INV),
        (dict(dout_strides=(1024, 132)), INV), (dict(workspace=None), WS),
        (dict(workspace_bytes=256), WS), (dict(workspace=P + 128), INV)]]
    + [(name, make, kw, code) for name, make in (("fa_qk_norm_rotary", _norm),
                                                 ("fa_qk_norm_rotary_backward", _norm_backward))
       for kw, code in [
        (dict(B=-1), INV), (dict(Hq=-1), INV), (dict(D=72), UNS), (dict(D=0), UNS),
        (dict(D=528, rot_dim=512), UNS), (dict(rot_dim=24), UNS), (dict(rot_dim=144), UNS),
        (dict(rot_dim=-16), UNS), (dict(dtype=fa.FA_E4M3), UNS), (dict(weight_dtype=fa.FA_FP16), UNS),
        (dict(amplitude=NAN), INV), (dict(eps=NAN), INV), (dict(eps=-1e-6), INV), (dict(eps=INF), INV),
        (dict(q=None), INV), (dict(k=P + 2), INV), (dict(q_strides=(1024, 132, 512)), INV),
        (dict(positions=None), INV), (dict(inv_freq=None), INV), (dict(positions=P + 2), INV),
        (dict(q_weight=P + 1), INV)]]
    + [("fa_qk_norm_rotary", _norm, kw, code) for kw, code in [
        (dict(q_out=None), INV), (dict(k_out_strides=(1024, 0, 512)), INV)]]
    + [("fa_qk_norm_rotary_backward", _norm_backward, kw, code) for kw, code in [
        (dict(dq_out=None), INV), (dict(dk_out=P + 8), INV), (dict(dq=None), INV),
        (dict(dk_strides=(1024, 0, 512)), INV), (dict(dq_weight=P + 2), INV),
        (dict(workspace=None), WS), (dict(workspace_bytes=128), WS), (dict(workspace=P + 16), INV)]]
    + [("gated_delta_step", _step, kw, code) for kw, code in [
        (dict(B=-1), INV), (dict(T=-1), INV), (dict(Hv=3), INV), (dict(Hk=0), INV),
        (dict(num_states=-1), INV), (dict(dk=64), UNS), (dict(dv=256), UNS),
        (dict(dtype=fa.FA_FP32), UNS), (dict(scale=NAN), INV), (dict(B=70000, num_states=70000), UNS),
        (dict(B=2), INV), (dict(states=None), INV), (dict(out=None), INV), (dict(g=None), INV),
        (dict(q=P + 8), INV), (dict(states=P + 4), INV), (dict(k_strides=(1024, 132, 512)), INV),
        (dict(out_strides=(1024, 0, 512)), INV), (dict(read_index=P + 2), INV)]]
)


@pytest.mark.parametrize("name,make,kw,code", CASES)
def test_refused(lib, name, make, kw, code):
    assert getattr(lib, name)(ctypes.byref(make(**kw)), None) == code
    assert fa.fa_last_error()


@pytest.mark.parametrize("name,make", [("fa_qk_norm_rotary", _norm), ("fa_qk_norm_rotary_backward", _norm_backward)])
@pytest.mark.parametrize("kw", [dict(Hq=65536), dict(Hk=2**31 - 1), dict(Hq=2**31 - 1, Hk=2**31 - 1),
                                dict(B=2**31 - 1, T=2**31 - 1)])
def test_norm_too_many_rows(lib, name, make, kw):
    """Counts whose sums or products would pass the integers that hold them."""
    assert getattr(lib, name)(ctypes.byref(make(**kw)), None) == UNS
    assert lib.fa_qk_norm_rotary_backward_workspace_size(ctypes.byref(_norm_backward(**kw))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(num_splits=-1), INV), (dict(num_splits=33), INV), (dict(num_splits=2), WS),
    (dict(num_splits=2, workspace=P, workspace_bytes=2 * 9 * 4 * 128 * 4), WS),
    (dict(num_splits=2, workspace=P + 16, workspace_bytes=1 << 20), INV),
    # 2^14 sequences, 2^13 kv heads and 32 parts: 2^32 work items
    (dict(num_splits=32, B=1 << 14, Hq=1 << 13, Hkv=1 << 13), UNS)])
def test_parts_refused(lib, kw, code):
    assert lib.fa_prefill_packed(ctypes.byref(_packed(**kw)), None) == code
    assert fa.fa_last_error()


def test_parts_workspace(lib):
    size = lambda **kw: lib.fa_packed_workspace_size(ctypes.byref(_packed(**kw)))  # noqa: E731
    assert size() == size(num_splits=1) == size(num_splits=33) == size(num_splits=2, total_q=0) == 0
    assert size(num_splits=3) >= 3 * 9 * 4 * (128 + 1) * 4
    # few query tiles and many keys: parts of eight tiles or more; many query tiles: none
    assert size(B=1, total_q=16, total_k=16384) >= 16 * 16 * 4 * (128 + 1) * 4
    assert size(B=1, total_q=16, total_k=2047) == size(B=1, total_q=16384, total_k=16384) == 0
    assert lib.fa_packed_workspace_size(None) == 0


@pytest.mark.parametrize("name", ["fa_prefill_packed", "fa_prefill_packed_backward", "fa_qk_norm_rotary",
                                  "fa_qk_norm_rotary_backward", "gated_delta_step"])
def test_null_struct(lib, name):
    assert getattr(lib, name)(None, None) == INV


def test_nothing_to_do(lib):
    """Empty calls are fine without any pointer."""
    none = dict(q=None, k=None, v=None, out=None)
    assert lib.fa_prefill_packed(ctypes.byref(_packed(B=0, **none)), None) == fa.FA_OK
    assert lib.fa_prefill_packed(ctypes.byref(_packed(total_q=0, **none)), None) == fa.FA_OK
    assert lib.fa_prefill_packed_backward(ctypes.byref(_packed_backward(total_q=0, total_k=0)), None) == fa.FA_OK
    assert lib.fa_qk_norm_rotary(ctypes.byref(_norm(T=0, q=None)), None) == fa.FA_OK
    assert lib.gated_delta_step(ctypes.byref(_step(B=0, states=None)), None) == fa.FA_OK


def test_workspace_sizes(lib):
    size = lib.fa_packed_backward_workspace_size
    # a word; 9 * 4 pairs of fp32; as many deltas of rows that see few keys; in pieces of 256
    assert size(ctypes.byref(_packed_backward())) == 256 + 512 + 256
    assert size(ctypes.byref(_packed_backward(total_q=1000))) == 256 + 32000 + 16128
    # fp16: a power of two a row, and a maximum for each 64 rows (D = 128) of a kv head
    assert size(ctypes.byref(_packed_backward(dtype=fa.FA_FP16))) == 256 + 512 + 256 + 256 + 256
    assert size(ctypes.byref(_packed_backward(total_q=1000, dtype=fa.FA_FP16))) == 256 + 32000 + 2 * 16128 + 256
    assert size(ctypes.byref(_packed_backward(B=0))) == 0
    assert size(ctypes.byref(_packed_backward(D=80))) == 0
    size = lib.fa_qk_norm_rotary_backward_workspace_size
    assert size(ctypes.byref(_norm_backward())) >= 2 * 128 * 4
    assert size(ctypes.byref(_norm_backward(T=0))) == 0
    assert size(ctypes.byref(_norm_backward(T=1 << 24))) < 1 << 22      # does not grow with the rows


def test_binding_refuses():
    """What the Python calls refuse by themselves: types, shapes, devices."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_prefill_packed(x, x, x, cu)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_qk_norm_rotary(x[None], None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        fa.gated_delta_step(x, x, x, x, x, x)
