"""Packed prompts without a device: pointers that no access may have, and the plan that the binding counts on."""
import ctypes

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
