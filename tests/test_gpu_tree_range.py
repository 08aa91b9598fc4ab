"""GPU checks of the tree attention at the ends of its ranges: cache values beyond the operand
type's, lengths and page ids out of range, scores that vanish, the longest sequence; against
the 64-bit evaluation of tests/_cache_ref.py."""
import math
import random

import pytest
import torch

import softmax_attention_gb300 as fa
from tests import _cache_ref as ref
from tests.test_gpu_tree import BF16, E4M3, FP16, Problem, pack, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def rows_at(x, i):
    return tuple(t[:, :, i] for t in x)


@pytest.mark.parametrize("dtype,byte", [(FP16, 135), (FP16, 150), (FP16, 254), (BF16, 247), (BF16, 254)])
@pytest.mark.parametrize("T,splits", [(4, 1), (24, 1), (24, 3), (70, 1)])
@pytest.mark.parametrize("chain", [True, False])
def test_hidden_values_beyond_the_operand_type(dtype, byte, T, splits, chain):
    """A drafted token whose V (code 448 times its scale) is beyond fp16, or beyond bf16: rows
    that do not see it are bit for bit what they are with its codes at zero."""
    pr = Problem(1, 4, 2, T, 128, 16, dtype, E4M3, [300])
    mask = torch.ones(T, T, dtype=torch.bool).tril() if chain else random_tree(T, random.Random(T))
    if not chain:
        mask[:, 2] = False
        mask[2, 2] = mask[T - 1, 2] = True
    hidden = ~mask[:, 2]
    at = 300 - T + 2
    pg, sl = int(pr.table[0, at // 16]), at % 16
    pr.vs[pg, :, sl] = byte
    pr.v[pg, :, sl] = 0
    words = None if chain else pack([mask], T).cuda()

    def call():
        args, kw = pr.gpu()
        return fa.fa_tree_decode_paged(*args, tree_mask=words, num_splits=splits, **kw)

    without = call()
    want = pr.want([T], [mask], 128 ** -0.5)
    pr.v[pg, :, sl, ::2] = 0x7E  # 448
    pr.v[pg, :, sl, 1::2] = 0xFE
    out, lse = call()
    i = hidden.cuda()
    assert torch.equal(out[:, :, i], without[0][:, :, i]) and torch.equal(lse, without[1])
    ref.check_tree(out[:, :, i], lse[:, :, i], rows_at(want, hidden), dtype, 128)


@pytest.mark.parametrize("T", [4, 24])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_largest_fp16_keys_and_values(T, D):
    """fp16's largest value in K and V, written by the library (stored as 256 * 2^8 = 65536):
    finite results, whether the token's weight counts, is negligible or is hidden."""
    g = torch.Generator().manual_seed(T + D)
    Hq, Hkv, ps, n = 4, 2, 16, 200
    P = -(-n // ps)
    k, v = (torch.randn(1, Hkv, n, D, generator=g) * 0.5 for _ in range(2))
    q = torch.randn(1, Hq, T, D, generator=g) * 0.5
    q[..., 3] = (torch.rand(1, Hq, T, generator=g) - 0.5) * 2.0 ** -10
    q[..., 5] = 4.0
    k[0, :, 11, 3] = 65504.0            # a key whose score is moderate
    v[0, :, 20] = 65504.0               # a value that counts
    k[0, :, 30, 5] = -40.0 * math.sqrt(D)   # a weight of about e^-160, with such a value
    v[0, :, 30, ::2] = -65504.0
    v[0, :, n - T + 1, 1::2] = 65504.0  # a drafted one, which row 0 does not see
    k[0, :, n - T + 1, 5] = -2.0 * math.sqrt(D)
    q, k, v = q.to(FP16), k.to(FP16), v.to(FP16)
    table = ref.make_table([n], ps, P, g).cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    kp = torch.zeros(P, Hkv, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    ks = torch.zeros(P, Hkv, ps, dtype=torch.uint8, device="cuda")
    vp, vs = kp.clone(), ks.clone()
    fa.fa_cache_append(k.cuda(), v.cuda(), kp, vp, table, lens, k_scales=ks, v_scales=vs)
    dk, dv = fa.fa_cache_gather(kp, vp, table, lens, n, dtype=torch.float32, k_scales=ks, v_scales=vs)
    assert dk.abs().max() == 65536 and dv.abs().max() == 65536
    out, lse = fa.fa_tree_decode_paged(q.cuda(), kp, vp, table, lens, n, k_scales=ks, v_scales=vs)
    rows = [[t[0].double().cpu().transpose(0, 1)] for t in (dk, dv)]
    want = ref.tree_attention(q, rows[0], rows[1], [T], None, D ** -0.5)
    assert want[0].abs().max() < 65504
    ref.check_tree(out, lse, want, FP16, D)


def test_seen_values_beyond_the_operand_type():
    """Seen by a row, a value beyond the fp16 operand counts as the operand's largest, 131008, in
    the 128-row kernel and as itself in the kernel for few rows."""
    for T, most in ((4, math.inf), (24, 131008.0)):
        pr = Problem(1, 4, 2, T, 128, 16, FP16, E4M3, [300])
        for t in (7, 299):  # of the context, and the last drafted token
            pg, sl = int(pr.table[0, t // 16]), t % 16
            pr.vs[pg, :, sl] = 139
            pr.v[pg, :, sl, ::2] = 0x7E   # 448 * 2^12
            pr.v[pg, :, sl, 1::2] = 0xC0  # -2 * 2^12
            pr.ks[pg, :, sl] = 127
            pr.k[pg, :, sl] = 0           # a weight of some 1 / 300
        args, kw = pr.gpu()
        out, lse = fa.fa_tree_decode_paged(*args, **kw)
        k, v = pr.rows(0)
        want = ref.tree_attention(pr.q, [k], [v.clamp(-most, most)], [T], None, 128 ** -0.5)
        assert want[0].abs().max() < 65504
        ref.check_tree(out, lse, want, FP16, 128, f"T={T}")


@pytest.mark.parametrize("dtype,cache", [(BF16, E4M3), (FP16, E4M3), (BF16, BF16)])
@pytest.mark.parametrize("T", [3, 20])
def test_bad_lengths_and_pages_of_both_kernels(dtype, cache, T):
    """Lengths and page ids out of range in the kernel for few rows and the 128-row one: the
    status is set, the sequences with a bad length are empty, a bad page stands for page 0 with
    its own scales (here outside what fp16 operands take for bf16 queries), the rest is as it was."""
    pr = Problem(4, 4, 2, T, 64, 16, dtype, cache, [40, 40, 40, 40])
    spare = next(i for i in range(1, pr.k.shape[0]) if not (pr.table == i).any())
    pr.table[pr.table == 0] = spare  # no sequence has page 0
    pr.v[0, :, (40 - T // 2) % 16, 3] = 0x7F if cache == E4M3 else math.nan  # of a drafted token, too
    if cache == E4M3:
        pr.vs[0, :, ::2] = 105
        if dtype == BF16:
            pr.vs[0, :, 1::2] = 150
    scale = 0.125
    (q, k, v, table, lens, L), kw = pr.gpu()
    good, _ = fa.fa_tree_decode_paged(q, k, v, table, lens, L, **kw)
    lens2 = lens.clone()
    lens2[1], lens2[2] = T - 1, 10 ** 6
    out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens2, L, **kw)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert not out[1:3].any() and (lse[1:3] == -math.inf).all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    lens2[1], lens2[2] = -1, -2 ** 31
    out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens2, L, **kw)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert not out[1:3].any() and torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    drafts = torch.tensor([T, T + 1, -1, 0], dtype=torch.int32).cuda()
    out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens, L, draft_lens=drafts, **kw)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert torch.equal(out[0], good[0]) and not out[1:].any() and (lse[1:] == -math.inf).all()
    for bad in (10 ** 6, -5, pr.k.shape[0]):
        table2 = table.clone()
        table2[1, 1] = table2[2, 2] = bad
        out, lse = fa.fa_tree_decode_paged(q, k, v, table2, lens, L, **kw)
        assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
        assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
        keep = pr.table.clone()
        pr.table[1, 1] = pr.table[2, 2] = 0
        ref.check_tree(out, lse, pr.want([T] * 4, None, scale), dtype, 64, f"page {bad}")
        pr.table = keep


@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_tiny_queries_and_score_scale(T, dtype):
    """Scores that vanish (q near 2^-105, or fp16's least, times a scale of 2^-45): every seen token
    weighs the same, hidden ones nothing."""
    pr = Problem(1, 4, 2, T, 128, 16, dtype, E4M3, [300])
    if dtype == BF16:
        pr.q = (pr.q.float() * 2.0 ** -105).to(BF16)
    else:
        pr.q = (pr.q.float() * 2.0 ** -20).to(FP16)
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, scale=2.0 ** -45, **kw)
    ref.check_tree(out, lse, pr.want([T], None, 2.0 ** -45), dtype, 128)


@pytest.mark.parametrize("T", [1, 20])
def test_the_longest_sequence(T):
    """max_pages * page_size as large as the call takes, over four pages that the table repeats:
    token counts next to 2^31 in both 8-bit kernels.  Keys of 0, so that every token weighs the same;
    V is 1, 2, 3 or 4 throughout a page.  Sums of such values are exact in fp32 here (a step of 16
    tokens adds a multiple of 2^11 below 2^33), so the output is the mean, rounded once after a
    merge of up to 608 parts (each of whose weights is off by 2^-19, its lse being near 2^4)."""
    ps, D = 64, 64
    pages = (2 ** 31 - 257) // ps
    n = pages * ps
    kp = torch.zeros(4, 1, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    vp = torch.arange(1, 5, device="cuda").view(4, 1, 1, 1).expand(4, 1, ps, D).to(torch.float32).to(E4M3).contiguous()
    ks = torch.full((4, 1, ps), 127, dtype=torch.uint8, device="cuda")
    table = (torch.arange(pages, dtype=torch.int32, device="cuda") % 4)[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, T, D, device="cuda").to(BF16)
    out, lse = fa.fa_tree_decode_paged(q, kp, vp, table, lens, n, k_scales=ks, v_scales=ks)
    torch.cuda.synchronize()
    assert (out.float() - 2.5).abs().max() <= 2.5 * (2.0 ** -8 + 2.0 ** -17)
    assert (lse.double() - math.log(n)).abs().max() <= 2.0 ** -17


def test_values_of_one_column_above_the_rest():
    """The kernel for few rows holds a weight times V's scale in fp16, relative to the row's largest
    such product.  A token of scale 2^9, zero but in one column, next to tokens of scale 2^-21 to
    2^-13: their columns keep an absolute error of 2^-32 of that product a unit of code.

    With w the weights, s the scales, c the codes, 2^ev = s: the running maximum of w s is at most
    the row's largest, and the fp16 weight of that maximum is 2^7, so the rounding (2^-11 of a
    weight, or 2^-25 where it is below 2^-14) is at most 2^-11 w_j s_j + 2^-32 max(w s)."""
    T, D, dtype = 2, 128, FP16
    pr = Problem(1, 4, 2, T, D, 16, dtype, E4M3, [300], scales=(106, 115))
    pr.ks[:] = 120
    pg, sl = int(pr.table[0, 2]), 5
    pr.vs[pg, :, sl] = 136
    pr.v[pg, :, sl] = 0
    pr.v[pg, :, sl, 9] = 0x38  # 1
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, num_splits=1, **kw)
    want = pr.want([T], None, D ** -0.5)
    o, l, mean_abs, reach, _ = want
    k, v = pr.rows(0)
    scales = torch.pow(2.0, ref.rows_of(pr.vs, pr.table, 0, 300).double() - 127.0)
    codes = (v / scales[..., None]).abs()
    half = 2.0 ** -11
    got = out.double().cpu()
    for h in range(4):
        for i in range(T):
            n = 300 - T + i + 1
            w = torch.softmax(k[:n, h // 2] @ pr.q[0, h, i].double() * D ** -0.5, 0)
            top = (w * scales[:n, h // 2]).max()
            delta = (D + 8) * 2.0 ** -23 * reach[0, h, i] + 2.0 ** -20
            bound = (half + 2 * delta) * mean_abs[0, h, i] + half * o[0, h, i].abs() + 2.0 ** -25 \
                + 2.0 ** -32 * top * codes[:n, h // 2].sum(0)
            assert ((got[0, h, i] - o[0, h, i]).abs() <= bound).all()
