"""Packed prompts at the ends of their range: long contexts, offsets that are broken beside ones that are
not, fp16 gradients over all of fp16's range, scores that are no number.  Against the plain 64-bit
references with derived bounds (tests/_packed_ref.py)."""
import math

import pytest
import torch

import softmax_attention_gb300 as fa
from tests import _packed_ref as ref
from tests.test_gpu_packed import BF, HF, Case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def _nan_workspace(size=1 << 24):
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ long contexts
@pytest.mark.parametrize("causal", [True, False])
def test_backward_of_a_context_past_the_product_with_the_group(causal):
    """One query of 128 heads over 20,000,000 keys: keys x heads of a group pass 2^31.  Keys and values repeat
    every 10,000 rows, so that each weight, and with it dk and dv, is that of one period over the repeats."""
    D, G, period, reps = 64, 128, 10000, 2000
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, G, D, generator=g).to(BF)
    base = torch.randn(period, 2, D, generator=g).to(BF)
    dout = torch.randn(1, G, D, generator=g).to(BF)
    scale = 0.125
    want = ref.attention(q, base[:, :1], base[:, 1:], False, scale, dout)  # (a single query sees every key)
    kv = base.cuda().repeat(reps, 1, 1)
    out = want["out"][0].to(BF).cuda()
    lse = (want["lse"][0] + math.log(reps)).float().cuda()
    cu, cuk = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (1, period * reps))
    _, dk, dv = fa.fa_prefill_packed_backward(dout.cuda(), q.cuda(), kv[:, :1], kv[:, 1:], out, lse, cu, cuk,
                                              causal=causal, scale=scale)
    torch.cuda.synchronize()
    for i in (0, 1, 320, 321, 322, 1000, 1677, 1678, reps - 1):
        at = slice(i * period, (i + 1) * period)
        for name, got in (("dk", dk), ("dv", dv)):
            value, bound = want[name]
            # (twice the bound: the exponent's rounding counts |lse|, and ln 2000 is not in it)
            ref.check(f"{name} of period {i}", got[at], value / reps, 2 * bound / reps)
