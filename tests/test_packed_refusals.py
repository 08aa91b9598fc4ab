"""Packed prompts without a device: pointers that no access may have, and the plan that the binding counts on."""
import ctypes
import random

import pytest

import softmax_attention_gb300 as fa
from tests.test_packed_abi import INV, P, _packed, _packed_backward, lib  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name,make,field", [
    ("fa_prefill_packed", _packed, "cu_seqlens_q"), ("fa_prefill_packed", _packed, "cu_seqlens_k"),
    ("fa_prefill_packed", _packed, "lse"), ("fa_prefill_packed_backward", _packed_backward, "cu_seqlens_q"),
    ("fa_prefill_packed_backward", _packed_backward, "cu_seqlens_k"),
    ("fa_prefill_packed_backward", _packed_backward, "lse")])
def test_misaligned(lib, name, make, field, off):  # noqa: F811
    """Offsets and lse are read and written four bytes at a time."""
    assert getattr(lib, name)(ctypes.byref(make(**{field: P + off})), None) == INV
    assert b"align" in lib.fa_last_error()


def test_parts_only_where_the_binding_looks_for_them(lib):  # noqa: F811
    """The binding asks for a workspace by itself only where the keys are 2048 a sequence or more: the plan has parts nowhere else."""
    rng = random.Random(5)
    parts = 0
    for _ in range(20000):
        Hkv, B = rng.choice([1, 2, 4, 8]), int(2 ** rng.uniform(0, 10))
        kw = dict(B=B, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 3, 8, 16, 128]), D=rng.choice([64, 128]),
                  total_q=int(2 ** rng.uniform(0, 17)), total_k=rng.choice([2048 * B - 1, 2048 * B, int(2 ** rng.uniform(0, 21))]))
        need = lib.fa_packed_workspace_size(ctypes.byref(_packed(num_splits=0, **kw)))
        assert need == 0 or kw["total_k"] >= 2048 * B, kw
        parts += need > 0
    assert parts > 1000
