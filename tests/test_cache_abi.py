"""Host-side checks of the serving-step calls (rotary positions, cache write and read, tree
attention): the host helpers against their formulas, and refusals: every bad argument is answered with its status code and a message before anything is enqueued, so no
device is needed."""
import ctypes
import math

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


def _tree(**kw):
    return _fill(fa.TreeArgs(), dict(
        q=P, q_strides=(2048, 512, 128), k_pages=P, v_pages=P, k_scales=P, v_scales=P, page_table=P,
        seq_lens=P, out=P, lse=P, B=1, Hq=4, Hkv=2, T=4, D=128, page_size=16, max_pages=4,
        num_pages=4, max_seq_len=64, mask_batches=1, scale=0.1, dtype=fa.FA_BF16,
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
    ("fa_tree_decode_paged", _tree, dict(T=-1), INV),
    ("fa_tree_decode_paged", _tree, dict(T=257), UNS),
    ("fa_tree_decode_paged", _tree, dict(Hq=5), INV),
    ("fa_tree_decode_paged", _tree, dict(Hq=258), UNS),
    ("fa_tree_decode_paged", _tree, dict(D=96), UNS),
    ("fa_tree_decode_paged", _tree, dict(dtype=fa.FA_FP32, cache_dtype=fa.FA_FP32), UNS),
    ("fa_tree_decode_paged", _tree, dict(cache_dtype=fa.FA_FP16), UNS),
    ("fa_tree_decode_paged", _tree, dict(page_size=4, max_pages=16), UNS),
    ("fa_tree_decode_paged", _tree, dict(page_size=256), UNS),
    ("fa_tree_decode_paged", _tree, dict(D=256, page_size=128), UNS),
    ("fa_tree_decode_paged", _tree, dict(max_seq_len=65), INV),
    ("fa_tree_decode_paged", _tree, dict(max_pages=1 << 27, num_pages=4), UNS),
    ("fa_tree_decode_paged", _tree, dict(num_pages=1 << 30), UNS),
    ("fa_tree_decode_paged", _tree, dict(scale=float("inf")), INV),
    ("fa_tree_decode_paged", _tree, dict(tree_mask=P, mask_batches=3), INV),
    ("fa_tree_decode_paged", _tree, dict(num_splits=-1), INV),
    ("fa_tree_decode_paged", _tree, dict(q=None), INV),
    ("fa_tree_decode_paged", _tree, dict(v_scales=None), INV),
    ("fa_tree_decode_paged", _tree, dict(k_scales=P + 4), INV),
    ("fa_tree_decode_paged", _tree, dict(out=P + 8), INV),
    ("fa_tree_decode_paged", _tree, dict(q_strides=(2048, 512, 4)), INV),
    ("fa_tree_decode_paged", _tree, dict(q_strides=(2048, 0, 128)), INV),
    ("fa_tree_decode_paged", _tree, dict(tree_mask=P + 4), INV),
    ("fa_tree_decode_paged", _tree, dict(num_splits=1, num_pages=0), INV),
    ("fa_tree_decode_paged", _tree, dict(num_splits=4, max_seq_len=1024, max_pages=64, T=16),
     fa.FA_ERR_WORKSPACE),
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
    ("fa_cache_gather", _gather, dict(B=0)), ("fa_tree_decode_paged", _tree, dict(B=0)),
    ("fa_tree_decode_paged", _tree, dict(T=0)),
])
def test_empty_work_needs_no_device(lib, name, make, kw):
    assert getattr(lib, name)(ctypes.byref(make(**kw)), None) == fa.FA_OK


@pytest.mark.parametrize("name", ["fa_rotary", "fa_cache_append", "fa_cache_gather",
                                  "fa_tree_decode_paged"])
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
    with pytest.raises(ValueError):
        fa.fa_tree_decode_paged(x, x, x, i, i[0, :1], 3)


def test_tree_workspace_is_that_of_the_plan(lib):
    """Split states of every row, and none unsplit or for sizes the call refuses."""
    def size(**kw):
        return lib.fa_tree_workspace_size(ctypes.byref(_tree(max_pages=64, max_seq_len=1024, **kw)))
    rows = 4 * 16
    assert size(num_splits=1) == 0
    assert size(T=16, num_splits=4) == rows * 4 * 128 * 4 + rows * 4 * 4
    assert size(T=16, num_splits=1000) == size(T=16, num_splits=8)  # 128-key tiles: 8 of them
    assert size(T=300) == 0 and size(B=0) == 0


@pytest.mark.parametrize("rot,base,factor,L", [(64, 10000.0, 8.0, 4096.0), (128, 500000.0, 32.0, 8192.0),
                                               (16, 10.0, 1.0, 100.0)])
def test_rotary_frequencies(lib, rot, base, factor, L):
    """Each scaling against its definition, evaluated here in fp64 (the library's and torch's powers
    are within a few units in the last place of each other)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    plain = torch.exp(-2.0 * i / rot * torch.log(torch.tensor(base, dtype=torch.float64)))

    def close(got, want):
        return ((got - want).abs() <= 1e-14 * want).all()

    f, amp = fa.rotary_frequencies(rot, base)
    assert close(f, plain) and amp == 1.0 and f[0] == 1.0
    f, amp = fa.rotary_frequencies(rot, base, "linear", factor)
    assert close(f, plain / factor) and amp == 1.0
    f, amp = fa.rotary_frequencies(rot, base, "base", factor)
    assert close(f[-1:], plain[-1:] / factor) and close(f[:1], plain[:1]) and amp == 1.0
    f, amp = fa.rotary_frequencies(rot, base, "by_parts", factor, L, 32.0, 1.0)
    turns = L * plain / (2 * torch.pi)
    assert close(f[turns >= 32], plain[turns >= 32])
    assert close(f[turns <= 1], plain[turns <= 1] / factor)
    mid = (turns > 1) & (turns < 32)
    g = (turns[mid] - 1) / 31
    assert ((f[mid] - plain[mid] * (g + (1 - g) / factor)).abs() <= 1e-13 * plain[mid]).all()
    assert abs(amp - (0.1 * math.log(factor) + 1)) <= 2 ** -23


@pytest.mark.parametrize("args", [
    (0,), (3,), (64, 1.0), (64, float("nan")), (64, 1e4, "linear", 0.5), (64, 1e4, "linear", float("nan")),
    (2, 1e4, "base", 2.0), (64, 1e4, "by_parts", 2.0, 0.0), (64, 1e4, "by_parts", 2.0, 100.0, 1.0, 1.0),
])
def test_rotary_frequencies_refusals(lib, args):
    with pytest.raises(fa.FAError) as e:
        fa.rotary_frequencies(*args)
    assert e.value.code == INV


def test_rotary_frequencies_unknown_scaling(lib):
    with pytest.raises(ValueError):
        fa.rotary_frequencies(64, scaling="other")
    assert lib.fa_rotary_frequencies(64, 1e4, 9, 1.0, 1.0, 2.0, 1.0, P, P) == INV


def test_tree_mask(lib):
    """Ancestors and self, for one tree and a batch, across words."""
    p = [-1, 0, 0, 1, -1, 4, 3]
    m = fa.tree_mask(p)
    assert m.shape == (1, 7, 1)
    assert m[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000, 0b1001011]
    chain = list(range(-1, 129))
    m = fa.tree_mask([chain, [-1] * 130])
    assert m.shape == (2, 130, 3)
    bits = ((m[..., None] >> torch.arange(64)) & 1).bool().flatten(2)[:, :, :130]
    i = torch.arange(130)
    assert torch.equal(bits[0], i[None, :] <= i[:, None]) and torch.equal(bits[1], torch.eye(130).bool())
    assert fa.tree_mask([]).shape == (1, 0, 0)
    for wrong in ([0], [-1, 1], [-2], [-1] * 257):
        with pytest.raises(fa.FAError):
            fa.tree_mask(wrong)
