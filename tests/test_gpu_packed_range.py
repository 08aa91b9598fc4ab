"""Packed prompts at the ends of their range: long contexts, offsets that are broken beside ones that are
not, fp16 gradients over all of fp16's range, scores that are no number or infinite.  Against the plain 64-bit
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


def test_a_work_item_of_seconds():
    """One query over 400,000,007 keys, unsplit: the waits for its last tile are longer than those of a pipeline that has
    stopped.  All scores are 0 but the last 128, of about 40 each: they alone count, as e^-40 x 4e8 is 1.7e-9."""
    D, n = 64, 400_000_007
    g = torch.Generator().manual_seed(7)
    last = (0.625 + 0.02 * torch.randn(128, 1, D, generator=g)).to(BF)
    kv = torch.zeros(n, 1, D, dtype=BF, device="cuda")
    kv[-128:] = last.cuda()
    q = torch.ones(1, 1, D, dtype=BF)
    cu, cuk = (torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in (1, n))
    out, lse = fa.fa_prefill_packed(q.cuda(), kv, kv, cu, cuk, scale=1.0, num_splits=1)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()
    want = ref.attention(q, last, last, False, 1.0)
    for name, got in (("out", out), ("lse", lse)):
        value, bound = want[name]
        ref.check(name, got, value, bound + 2e-9)


# ------------------------------------------------------------------ broken offsets
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("offsets,first,end", [
    ([0, 64, 32], 0, 64), ([-5, 64, 128], 64, 128), ([0, 64, 129], 0, 64), ([100, 0, 64], 0, 64),
    ([0, 90, 3, 2], 0, 90), ([0, 100, 2 ** 31 - 1], 0, 100), ([128, 128, 5, 100, 0], 5, 100)])
def test_gradients_beside_broken_offsets(offsets, first, end, dtype):
    """A sequence whose offsets hold has its gradients, whatever stands beside it; other rows stay as they were."""
    c = Case([128], 4, 2, 64, dtype, seed=17)
    q, k, v = c.gpu()
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = torch.full((128, 4, 64), NAN, dtype=dtype, device="cuda")
    lse = torch.full((128, 4), NAN, device="cuda")
    fa.fa_prefill_packed(q, k, v, cu, scale=0.125, out=out, lse=lse)
    dq = torch.full_like(out, 7.0)
    dk, dv = (torch.full((128, 2, 64), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    do = c.do.clone()
    do[:first], do[end:] = NAN, NAN
    fa.fa_prefill_packed_backward(do.cuda(), q, k, v, out, lse, cu, scale=0.125, dq=dq, dk=dk, dv=dv,
                                  workspace=_nan_workspace())
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    at = slice(first, end)
    want = ref.attention(*(t[at] for t in c.cpu()), True, 0.125, c.do[at])
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, t[at], *want[name])
        assert (t[:first] == 7).all() and (t[end:] == 7).all()


# ------------------------------------------------------------------ fp16 gradients
def _check_half(got, q, k, v, dout, causal, scale):
    """Gradients of one sequence.  dS is held times a power of two that brings the largest sum |dout_i| max |v| (of the
    row for dq, of the sequence's rows for dk) to 2^14 or more: half the least subnormal over that power, 2^-25 / f
    with f >= 2^14 / (sum |dout_i| max |v|), in place of the reference's, which knows |dout| alone."""
    want = ref.attention(q, k, v, causal, scale, dout)
    n, Hq, D = q.shape
    m, Hkv = k.shape[:2]
    G = Hq // Hkv
    sums = dout.double().abs().sum(-1)                                              # [n,Hq]
    top = v.double().abs().amax((0, 2)).repeat_interleave(G)                        # [Hq]
    step = 2.0 ** -25 * sums * top / 2.0 ** 14                                      # of a row
    seen = ref._visible(n, m, causal).double()
    kk = k.double().abs().repeat_interleave(G, 1)
    more = abs(scale) * step[..., None] * torch.einsum("ij,jhd->ihd", seen, kk)
    value, bound = want["dq"]
    ref.check("dq", got[0], value, bound + more)
    of_all = step.view(n, Hkv, G).amax((0, 2))                                      # of the sequence and kv head
    rows = torch.einsum("ij,ihd->jhd", seen, q.double().abs()).view(m, Hkv, G, D).sum(2)
    value, bound = want["dk"]
    ref.check("dk", got[1], value, bound + abs(scale) * of_all[None, :, None] * rows)
    ref.check("dv", got[2], *want["dv"])


@pytest.mark.parametrize("size,big", [(0.0019, 100.0), (1.0, 150.0), (1.0, 1000.0), (2.0 ** -20, 60000.0), (16.0, 0.01)])
@pytest.mark.parametrize("D", [64, 128])
def test_half_gradients_of_large_values(D, size, big):
    """Values aligned with dout: dP = +- D size big, whose products with the power of two have to stay in range.
    (q and k are small, and so are the gradients.)"""
    lens = [2, 40, 200]
    c = Case(lens, 4, 2, D, HF, seed=5)
    c.x[:, :6] *= 2.0 ** -6
    sign = torch.where(torch.arange(c.x.shape[0]) % 2 == 0, 1.0, -1.0)[:, None, None]
    c.x[:, 6:] = (sign * big * (1 + 0.1 * c.x[:, 6:].float().clamp(-0.9, 0.9))).to(HF)
    c.do = torch.full_like(c.do, size)
    scale = 1.0 / D
    for causal in (True, False):
        q, k, v = c.gpu()
        out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), causal=causal, scale=scale)
        got = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), causal=causal,
                                            scale=scale, workspace=_nan_workspace())
        for a, b in zip(c.cu, c.cu[1:]):
            _check_half([t[a:b] for t in got], *(t[a:b] for t in c.cpu()), c.do[a:b], causal, scale)


def test_half_gradient_of_two_keys():
    """The smallest such call: one query, two keys of equal weight, v = +100 and -100, dout 0.0019 in every column."""
    D = 128
    q = torch.full((1, 1, D), 2.0 ** -7, dtype=HF)
    k = torch.full((2, 1, D), 2.0 ** -7, dtype=HF)
    v = torch.tensor([100.0, -100.0]).view(2, 1, 1).expand(2, 1, D).to(HF).contiguous()
    do = torch.full((1, 1, D), 0.0019, dtype=HF)
    cu, cuk = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda()
    out, lse = fa.fa_prefill_packed(q.cuda(), k.cuda(), v.cuda(), cu, cuk, causal=False, scale=0.1)
    got = fa.fa_prefill_packed_backward(do.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, cu, cuk, causal=False, scale=0.1)
    _check_half(got, q, k, v, do, False, 0.1)


@pytest.mark.parametrize("small,large", [(0.01, 1000.0), (0.0, 60000.0), (1.0, 300.0)])
@pytest.mark.parametrize("D,G,causal", [(64, 2, True), (128, 1, False), (128, 4, True)])
def test_half_gradients_of_values_that_differ_by_tile(D, G, causal, small, large):
    """Keys of small values in one tile, of large ones in others: delta, a mean over all of them, is far larger than the
    dP of the small ones, in their dS too."""
    L = 500
    c = Case([L, 40], 2 * G, 2, D, HF, seed=29)
    c.x[:, :2 * G + 2] *= 2.0 ** -6
    size = torch.full((c.x.shape[0], 1, 1), large)
    size[:100], size[200:390] = small, small
    c.x[:, 2 * G + 2:] = (size * (1 + 0.1 * c.x[:, 2 * G + 2:].float().clamp(-0.9, 0.9))).to(HF)
    c.do = torch.full_like(c.do, 2.0 ** -6)
    scale = 1.0 / D
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), causal=causal, scale=scale)
    got = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), causal=causal, scale=scale,
                                        workspace=_nan_workspace())
    for a, b in zip(c.cu, c.cu[1:]):
        _check_half([t[a:b] for t in got], *(t[a:b] for t in c.cpu()), c.do[a:b], causal, scale)


# ------------------------------------------------------------------ samples of a pack
@pytest.mark.parametrize("lens", [[150, 150], [70, 1, 133, 40], [64, 128, 5]])
@pytest.mark.parametrize("D", [64, 128])
def test_half_gradients_of_a_sample_are_its_own(D, lens):
    """Samples whose dout, and whose values, are powers of two apart, and one of infinities: each has the bits of the same sample
    packed alone, and is inside bounds that know nothing of the others."""
    c = Case(lens, 8, 2, D, HF, seed=23)
    sizes = [2.0 ** 12, 2.0 ** -8, 1.0, 2.0 ** -12]
    for i, (a, b) in enumerate(zip(c.cu, c.cu[1:])):
        c.do[a:b] = (c.do[a:b].float() * sizes[i % 4]).to(HF)
        c.x[a:b, 10:] = (c.x[a:b, 10:].float() * sizes[(i + 1) % 4]).to(HF)
    scale = 1.0 / math.sqrt(D)
    for infinite in (False, True):
        do = c.do.clone()
        if infinite:
            do[c.cu[1] - 1, 0, 0] = INF  # of the first sample
        q, k, v = c.gpu()
        out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale)
        got = fa.fa_prefill_packed_backward(do.cuda(), q, k, v, out, lse, *c.offsets(), scale=scale)
        for i, (a, b) in enumerate(zip(c.cu, c.cu[1:])):
            if infinite and i == 0:
                continue
            one = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
            alone = fa.fa_prefill_packed_backward(do[a:b].cuda(), q[a:b], k[a:b], v[a:b], out[a:b], lse[a:b], one,
                                                  scale=scale)
            for name, x, y in zip(("dq", "dk", "dv"), got, alone):
                assert torch.equal(x[a:b], y), (name, i)
            _check_half([t[a:b] for t in got], *(t[a:b] for t in c.cpu()), do[a:b], True, scale)


# ------------------------------------------------------------------ scores that are no number
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
@pytest.mark.parametrize("splits", [1, 3])
def test_a_nan_score_reaches_lse(D, dtype, splits):
    """A NaN in a key: out and lse of every row that sees it are NaN, the others' as ever."""
    for at in (0, 37, 200, 389):
        c = Case([90], 4, 2, D, dtype, klens=[390], seed=19)
        c.y[at, :2, 5] = NAN
        q, k, v = c.gpu()
        out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=0.1, num_splits=splits)
        clean = Case([90], 4, 2, D, dtype, klens=[390], seed=19)
        want = next(clean.want(True, 0.1))[2]
        n = max(0, min(90, at - 300))  # rows in front of the key
        assert out[n:].isnan().all() and lse[n:].isnan().all()
        ref.check("out", out[:n], *(t[:n] for t in want["out"]))
        ref.check("lse", lse[:n], *(t[:n] for t in want["lse"]))


# ------------------------------------------------------------------ infinite scores
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("hidden", [20, 40, 150])
def test_scores_of_minus_infinity(hidden, splits, causal):
    """Keys of which a column is -inf, in front of keys with scores far below 0: weights of 0, and no bearing on the rest."""
    L, D = 400, 64
    c = Case([L], 2, 1, D, HF, seed=6)
    c.x[:, :2, 0] = 8.0
    c.x[:, 2, 0] = -100.0
    clean = c.x.clone()
    c.x[:hidden, 2, 0] = -INF
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), causal=causal, scale=1.0, num_splits=splits)
    # rows from `hidden` on: what the other keys alone give
    q, k, v = c.views(clean[hidden:], None)
    want = ref.attention(q, k, v, causal, 1.0)
    for name, got in (("out", out), ("lse", lse)):
        ref.check(name, got[hidden:], *want[name])
