"""GPU checks of the tree attention over a paged cache against a plain 64-bit evaluation, query
by query, that leaves hidden keys out altogether (tests/_cache_ref.py)."""
import math
import random

import pytest
import torch

import softmax_attention_gb300 as fa
from tests import _cache_ref as ref
from tests._guard import Guarded

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def random_tree(T, rng):
    """Boolean [T,T]: each token's ancestors and itself; a parent is any earlier token or the
    context."""
    m = torch.zeros(T, T, dtype=torch.bool)
    for i in range(T):
        p = rng.randrange(-1, i)
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def pack(masks, T):
    """int64 words [len(masks), T, ceil(T/64)] of boolean [T,T] masks."""
    out = []
    for m in masks:
        rows = []
        for i in range(T):
            v = sum(1 << j for j in range(T) if m[i, j])
            words = [(v >> (64 * w)) & (2 ** 64 - 1) for w in range(-(-T // 64))]
            rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in words])
        out.append(rows)
    return torch.tensor(out, dtype=torch.int64)


class Problem:
    """A pool, a page table and queries on the CPU; pages of 16-bit values, or 8-bit codes."""

    def __init__(self, B, Hq, Hkv, T, D, ps, dtype, cache, lens, seed=0, scales=(118, 124), sigma=1.0):
        g = torch.Generator().manual_seed(seed + 7 * T + D)
        self.dtype, self.cache, self.lens, self.D, self.T = dtype, cache, lens, D, T
        P = sum(-(-n // ps) for n in lens) + 2
        self.table = ref.make_table(lens, ps, P, g)
        shape = (P, Hkv, ps, D)
        if cache == E4M3:
            self.k, self.v = ((torch.randn(shape, generator=g) * 90).clamp(-448, 448).to(E4M3).view(torch.uint8)
                              for _ in range(2))
            self.ks, self.vs = (torch.randint(*scales, shape[:3], generator=g, dtype=torch.uint8)
                                for _ in range(2))
        else:
            self.k, self.v = ((torch.randn(shape, generator=g) * 0.7).to(dtype) for _ in range(2))
            self.ks = self.vs = None
        self.q = (torch.randn(B, Hq, T, D, generator=g) * sigma).to(dtype)

    def rows(self, b):
        out = []
        for pages, scales in ((self.k, self.ks), (self.v, self.vs)):
            r = ref.rows_of(pages, self.table, b, self.lens[b])
            out.append(r.double() if scales is None
                       else ref.dequantise(r, ref.rows_of(scales, self.table, b, self.lens[b])))
        return out

    def want(self, draft_lens, masks, scale):
        k, v = zip(*(self.rows(b) for b in range(len(self.lens))))
        return ref.tree_attention(self.q, k, v, draft_lens, masks, scale)

    def gpu(self):
        k, v = self.k.cuda(), self.v.cuda()
        if self.cache == E4M3:
            k, v = k.view(E4M3), v.view(E4M3)
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        kw = {} if self.ks is None else dict(k_scales=self.ks.cuda(), v_scales=self.vs.cuda())
        return (self.q.cuda(), k, v, self.table.cuda(), lens, max(self.lens)), kw


CASES = [
    # B, Hq, Hkv, T, D, page, lens, draft lens, masked, splits
    (1, 4, 1, 1, 128, 16, [1], None, False, 0),
    (2, 8, 2, 1, 128, 16, [300, 17], None, False, 0),
    (1, 4, 2, 7, 64, 8, [7], None, True, 0),                    # no context
    (3, 8, 8, 5, 128, 32, [128, 129, 5], None, True, 0),        # a tile edge at the tree's end
    (2, 12, 4, 16, 128, 16, [515, 140], [16, 3], True, 0),      # three heads a group, padding
    (1, 8, 1, 33, 256, 64, [333], None, True, 0),
    (2, 5, 1, 64, 64, 64, [200, 64], [64, 1], True, 3),         # forced split
    (1, 4, 4, 65, 128, 16, [400], None, True, 0),               # two mask words
    (1, 2, 1, 130, 64, 128, [260], None, True, 2),              # three, across a tile edge
    (1, 2, 2, 256, 128, 8, [300], None, True, 0),               # the largest tree
    (1, 8, 1, 40, 128, 16, [700], None, False, 0),              # a chain, several query tiles
    (3, 4, 2, 4, 256, 8, [70, 4, 9], [4, 0, 2], True, 0),       # a sequence without a query
    (1, 128, 1, 2, 64, 16, [90], None, True, 0),                # one query a tile
    (1, 7, 1, 3, 128, 128, [1100], None, True, 0),              # split by the library
    (2, 4, 4, 3, 64, 128, [700, 3], None, True, 0),             # few rows, pages of four slices
    (1, 16, 1, 1, 256, 8, [515], None, False, 0),               # sixteen rows, two pages a slice
    (2, 8, 2, 4, 128, 64, [129, 70], [2, 4], True, 2),          # sixteen rows, split, padding
    (3, 2, 1, 1, 128, 32, [1, 32, 33], None, False, 0),         # lengths around a slice
    (2, 8, 8, 1, 64, 8, [0, 700], None, False, 0),              # an empty sequence
    (1, 6, 2, 5, 256, 32, [1000], None, True, 5),               # fifteen rows, D = 256, split
]


@pytest.mark.parametrize("dtype,cache", [(BF16, E4M3), (FP16, E4M3), (BF16, BF16), (FP16, FP16)])
@pytest.mark.parametrize("B,Hq,Hkv,T,D,ps,lens,drafts,masked,splits", CASES)
def test_parity(B, Hq, Hkv, T, D, ps, lens, drafts, masked, splits, dtype, cache):
    if D == 256 and ps > 64:
        pytest.skip("page size")
    rng = random.Random(T)
    pr = Problem(B, Hq, Hkv, T, D, ps, dtype, cache, lens)
    masks = [random_tree(T, rng) for _ in range(B)] if masked else None
    scale = 1.0 / math.sqrt(D)
    args, kw = pr.gpu()
    og, lg = Guarded((B, Hq, T, D), dtype), Guarded((B, Hq, T), torch.float32)
    fa.fa_tree_decode_paged(*args, tree_mask=pack(masks, T).cuda() if masked else None, scale=scale,
                            draft_lens=None if drafts is None else torch.tensor(drafts, dtype=torch.int32).cuda(),
                            num_splits=splits, out=og.view, lse=lg.view, **kw)
    torch.cuda.synchronize()
    og.assert_intact("out")
    lg.assert_intact("lse")
    want = pr.want(drafts or [T] * B, masks, scale)
    ref.check_tree(og.view, lg.view, want, dtype, D, f"{lens} T={T}")


@pytest.mark.parametrize("cache", [E4M3, BF16])
def test_shared_mask_and_strided_queries(cache):
    """One mask for the whole batch; queries as a projection leaves them ([B,T,H,D])."""
    B, Hq, Hkv, T, D, ps, lens = 3, 8, 2, 6, 128, 16, [40, 6, 133]
    pr = Problem(B, Hq, Hkv, T, D, ps, BF16, cache, lens)
    mask = random_tree(T, random.Random(1))
    (q, *rest), kw = pr.gpu()
    wide = torch.zeros(B, T, Hq + 4, D, dtype=BF16, device="cuda")
    wide[:, :, 2:2 + Hq] = q.transpose(1, 2)
    out, lse = fa.fa_tree_decode_paged(wide[:, :, 2:2 + Hq].transpose(1, 2), *rest,
                                       tree_mask=pack([mask], T).cuda(), **kw)
    want = pr.want([T] * B, [mask] * B, D ** -0.5)
    ref.check_tree(out, lse, want, BF16, D)


@pytest.mark.parametrize("cache", [E4M3, BF16])
@pytest.mark.parametrize("T", [3, 70])
def test_empty_rows(cache, T):
    """Mask rows without a bit: empty when there is no context, context only otherwise; a row
    that does not see itself."""
    pr = Problem(2, 4, 2, T, 64, 16, BF16, cache, [T, T + 50])
    m = torch.zeros(T, T, dtype=torch.bool)
    m[1, 0] = True          # sees its parent, not itself
    m[2] = torch.arange(T) <= 2
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, tree_mask=pack([m], T).cuda(), **kw)
    want = pr.want([T, T], [m, m], 0.125)
    assert (want[1][0, :, 0] == -math.inf).all() and torch.isfinite(want[1][1]).all()
    ref.check_tree(out, lse, want, BF16, 64)


@pytest.mark.parametrize("dtype,cache", [(BF16, E4M3), (BF16, BF16), (FP16, FP16), (FP16, E4M3)])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("T", [4, 24])
def test_hidden_values_do_not_leak(dtype, cache, splits, T):
    """NaN and infinities in one branch's keys and values: rows that do not see the branch are
    as if it were not there, rows that do are what the formula says; slots past the sequence's
    end hold NaN too."""
    lens, ps, D = [300, T + 1], 16, 128
    pr = Problem(2, 4, 2, T, D, ps, dtype, cache, lens)
    rng = random.Random(9)
    mask = random_tree(T, rng)
    mask[:, 1] = False      # token 1 is seen by row 1 and row T-1 alone
    mask[1, 1] = mask[T - 1, 1] = True
    mask[:, 2] = False      # token 2 by row 2 alone
    mask[2, 2] = True
    nan = 0x7F if cache == E4M3 else math.nan
    inf = 0xFF if cache == E4M3 else math.inf
    for b, n in enumerate(lens):
        def at(t):
            return int(pr.table[b, t // ps]), t % ps
        pg, sl = at(n - T + 1)
        pr.v[pg, :, sl, 5] = nan
        pr.v[pg, 0, sl, 77] = inf
        pg, sl = at(n - T + 2)
        pr.k[pg, 1, sl, 3] = nan
        if n % ps:  # the rest of the last page
            pg = int(pr.table[b, (n - 1) // ps])
            pr.k[pg, :, n % ps:] = nan
            pr.v[pg, :, n % ps:] = nan
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, tree_mask=pack([mask], T).cuda(), num_splits=splits, **kw)
    k, v = zip(*(pr.rows(b) for b in range(2)))
    want = ref.tree_attention(pr.q, k, v, [T, T], [mask] * 2, D ** -0.5)
    o, l = want[0], want[1]
    # the reference's own NaN rows: value columns 5 (and 77) of rows 1 and T-1, all of row 2 of
    # the heads of kv head 1
    assert torch.isnan(o[:, :, 1, 5]).all() and torch.isnan(o[:, 2:, 2]).all()
    assert torch.isfinite(o[:, :, 0]).all()
    got, gl = out.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(o))
    assert torch.equal(torch.isinf(got), torch.isinf(o)) and torch.equal(got[torch.isinf(o)], o[torch.isinf(o)])
    assert torch.equal(torch.isnan(gl), torch.isnan(l))
    fin = torch.isfinite(o)
    clean = (torch.where(fin, o, 0.0), torch.where(torch.isnan(l), 0.0, l),
             torch.where(fin, want[2], 0.0), torch.nan_to_num(want[3]),
             torch.where(fin, want[4], 0.0))
    ref.check_tree(torch.where(fin, got, 0.0), torch.where(torch.isnan(l), 0.0, gl), clean, dtype, D)


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 16), (256, 64)])
@pytest.mark.parametrize("cache", [E4M3, BF16])
def test_running_max_rises_every_tile(D, ps, cache):
    """Scores that grow along the keys by about 12 (log2 units) a KV tile: every tile moves the
    running maximum past the lazy rescale's threshold."""
    T, n = 9, 1100
    pr = Problem(2, 8, 2, T, D, ps, BF16, cache, [n, 700])
    bn = 64 if D == 256 else 128
    slope = 12.0 / (bn * 1.4426950408889634)  # natural log units a key, over scale
    pr.q[..., 0] = 4.0
    for b, L in enumerate(pr.lens):
        for t in range(L):
            pg, sl = int(pr.table[b, t // ps]), t % ps
            val = slope * t * math.sqrt(D) / 4.0
            if cache == E4M3:
                pr.ks[pg, :, sl] = 124 if val < 50 else 128  # 2^-3 or 2
                s = 2.0 ** (int(pr.ks[pg, 0, sl]) - 127)
                pr.k[pg, :, sl, 1:] = 0
                pr.k[pg, :, sl, 0] = torch.tensor(val / s).clamp(max=448).to(E4M3).view(torch.uint8)
            else:
                pr.k[pg, :, sl, 0] = val
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, num_splits=1, **kw)
    ref.check_tree(out, lse, pr.want([T] * 2, None, D ** -0.5), BF16, D)


@pytest.mark.parametrize("dtype,lo,hi", [(BF16, 1, 240), (FP16, 112, 134)])
@pytest.mark.parametrize("T", [1, 20])
def test_wide_row_scales(dtype, lo, hi, T):
    """Scale bytes over the whole range (bf16: far beyond fp16's, and past the exponent where the
    widening takes two products), and every e4m3 code."""
    pr = Problem(1, 4, 2, T, 128, 16, dtype, E4M3, [257])
    g = torch.Generator().manual_seed(4)
    pr.vs = torch.randint(lo, hi, pr.vs.shape, generator=g, dtype=torch.uint8)
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]
    pr.v = codes[torch.randint(0, codes.numel(), pr.v.shape, generator=g)]
    if dtype == BF16:
        # keys scaled up and down by the same large powers, queries so that scores stay O(1)
        pr.ks = torch.where(torch.rand(pr.ks.shape, generator=g) < 0.5, 150, 135).to(torch.uint8)
        pr.q = (pr.q.float() * 2.0 ** -30).to(BF16)
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, **kw)
    ref.check_tree(out, lse, pr.want([T], None, 128 ** -0.5), dtype, 128)


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
@pytest.mark.parametrize("cache", [E4M3, BF16])
def test_scales_of_scores(scale, cache):
    pr = Problem(1, 4, 1, 5, 128, 16, BF16, cache, [150])
    mask = random_tree(5, random.Random(2))
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, tree_mask=pack([mask], 5).cuda(), scale=scale, **kw)
    ref.check_tree(out, lse, pr.want([5], [mask], scale), BF16, 128)


def test_many_sequences():
    """More sequences than the kernel ranks by length (each then keeps its index)."""
    B = 400
    lens = [1 + (37 * i) % 90 for i in range(B)]
    for cache in (E4M3, BF16):
        pr = Problem(B, 2, 1, 1, 64, 8, BF16, cache, lens)
        args, kw = pr.gpu()
        out, lse = fa.fa_tree_decode_paged(*args, **kw)
        ref.check_tree(out, lse, pr.want([1] * B, None, 0.125), BF16, 64)


def test_matches_paged_decode_and_prefill():
    """One token over a 16-bit cache is the paged decode; a chain is the causal paged prefill."""
    pr = Problem(3, 8, 2, 12, 128, 16, BF16, BF16, [500, 12, 129])
    (q, k, v, table, lens, L), _ = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens, L)
    o2, l2 = fa.fa_prefill_paged(q, k, v, table, lens, L, causal=True)
    assert torch.allclose(lse, l2, atol=1e-5) and (out.float() - o2.float()).abs().max() <= 2 ** -7
    out, lse = fa.fa_tree_decode_paged(q[:, :, -1:].contiguous(), k, v, table, lens, L)
    o2, l2 = fa.fa_decode_paged(q[:, :, -1].contiguous(), k, v, table, lens, L)
    assert torch.allclose(lse[..., 0], l2, atol=1e-5)
    assert (out[:, :, 0].float() - o2.float()).abs().max() <= 2 ** -7


@pytest.mark.parametrize("cache", [E4M3, BF16])
def test_no_key_at_all(cache):
    """max_seq_len 0: only empty rows; and nothing to do."""
    q = torch.randn(2, 4, 3, 64, device="cuda").to(BF16)
    pages = torch.zeros(1, 2, 16, 64, device="cuda").to(cache)
    kw = {}
    if cache == E4M3:
        kw = dict(k_scales=torch.full((1, 2, 16), 127, dtype=torch.uint8, device="cuda"))
        kw["v_scales"] = kw["k_scales"]
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = fa.fa_tree_decode_paged(q, pages, pages, table, lens, 0, **kw)
    assert not out.any() and (lse == -math.inf).all()
    out, lse = fa.fa_tree_decode_paged(q[:, :, :0], pages, pages, table, lens, 16, **kw)
    assert out.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)


@pytest.mark.parametrize("cache", [E4M3, BF16])
@pytest.mark.parametrize("T", [2, 40])
def test_padding_queries_hold_anything(cache, T):
    """NaN in the queries of padding rows (at and past draft_lens) stays there: those rows are
    empty, every other row as without it."""
    pr = Problem(2, 8, 2, T, 128, 16, BF16, cache, [300, 77])
    (q, *rest), kw = pr.gpu()
    drafts = torch.tensor([1, T - 1], dtype=torch.int32, device="cuda")
    good = fa.fa_tree_decode_paged(q, *rest, draft_lens=drafts, **kw)
    q[0, :, 1:] = math.nan
    q[1, :, T - 1:] = math.inf
    out, lse = fa.fa_tree_decode_paged(q, *rest, draft_lens=drafts, **kw)
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    assert not out[0, :, 1:].any() and (lse[0, :, 1:] == -math.inf).all()


def test_a_cache_past_four_gigabytes():
    """Pages whose byte offsets pass 32 bits: written, read back and attended there."""
    Hkv, ps, D, T = 8, 64, 128, 20
    P = (1 << 32) // (Hkv * ps * D) + 40
    kp = torch.empty(P, Hkv, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    vp = torch.empty(P, Hkv, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    ks = torch.empty(P, Hkv, ps, dtype=torch.uint8, device="cuda")
    vs = torch.empty(P, Hkv, ps, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(5)
    n = 200
    table = torch.tensor([[P - 1, 3, P - 30, P - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 1, Hkv, n, D, generator=g).to(BF16)
    fa.fa_cache_append(x[0].cuda(), x[1].cuda(), kp, vp, table, lens, k_scales=ks, v_scales=vs)
    k, v = fa.fa_cache_gather(kp, vp, table, lens, n, dtype=torch.float32, k_scales=ks, v_scales=vs)
    for got, src in ((k, x[0]), (v, x[1])):
        want = ref.dequantise(*ref.quantise(src.float()))
        assert torch.equal(got.cpu().double(), want)
    rows = [[t[0].double().cpu().transpose(0, 1)] for t in (k, v)]
    for t in (1, T):  # the kernel for few rows, and the 128-row one
        q = torch.randn(1, 8, t, D, generator=g).to(BF16)
        out, lse = fa.fa_tree_decode_paged(q.cuda(), kp, vp, table, lens, n, k_scales=ks, v_scales=vs)
        want = ref.tree_attention(q, rows[0], rows[1], [t], None, D ** -0.5)
        ref.check_tree(out, lse, want, BF16, D)


def test_bad_lengths_and_pages():
    pr = Problem(4, 4, 2, 3, 64, 16, BF16, E4M3, [40, 40, 40, 40])
    (q, k, v, table, lens, L), kw = pr.gpu()
    good, _ = fa.fa_tree_decode_paged(q, k, v, table, lens, L, **kw)
    lens2 = lens.clone()
    lens2[1], lens2[2] = 2, 10 ** 6     # fewer tokens than drafted; more than the table holds
    out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens2, L, **kw)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert not out[1:3].any() and (lse[1:3] == -math.inf).all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    drafts = torch.tensor([3, 4, -1, 0], dtype=torch.int32).cuda()
    out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens, L, draft_lens=drafts, **kw)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert torch.equal(out[0], good[0]) and not out[1:].any()
    table2 = table.clone()
    table2[1, 1] = 10 ** 6
    out, lse = fa.fa_tree_decode_paged(q, k, v, table2, lens, L, **kw)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert torch.equal(out[0], good[0]) and torch.isfinite(out.float()).all()


def test_a_speculative_step():
    """The operators together, as a serving step uses them: rotate the drafted queries and keys
    at their depths, write the keys and values into an 8-bit cache that holds the context, attend
    the tree; against 64-bit attention over what was read back, and against the whole in 64 bits."""
    g = torch.Generator().manual_seed(21)
    B, Hq, Hkv, T, D, ps = 2, 8, 2, 9, 128, 16
    ctx = [100, 37]
    lens = [c + T for c in ctx]
    P = sum(-(-n // ps) for n in lens)
    table = ref.make_table(lens, ps, P, g)
    f = 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64)
    kp = torch.zeros(P, Hkv, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    vp = kp.clone()
    ks = torch.zeros(P, Hkv, ps, dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    hist = torch.randn(2, B, Hkv, max(ctx), D, generator=g).to(BF16)
    td, ld = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    fa.fa_cache_append(hist[0].cuda(), hist[1].cuda(), kp, vp, td, torch.tensor(ctx, dtype=torch.int32).cuda(),
                       new_lens=torch.tensor(ctx, dtype=torch.int32).cuda(), k_scales=ks, v_scales=vs,
                       inv_freq=f.cuda())
    mask = random_tree(T, random.Random(3))
    depth = mask.sum(1) - 1
    pos = torch.stack([c + depth for c in ctx]).to(torch.int32)
    q = torch.randn(B, Hq, T, D, generator=g).to(BF16)
    kv = torch.randn(2, B, Hkv, T, D, generator=g).to(BF16)

    def step():
        qr, _ = fa.fa_rotary(q.cuda(), None, pos.cuda(), f.cuda())
        fa.fa_cache_append(kv[0].cuda(), kv[1].cuda(), kp, vp, td, ld, k_scales=ks, v_scales=vs,
                           inv_freq=f.cuda(), positions=pos.cuda())
        out, lse = fa.fa_tree_decode_paged(qr, kp, vp, td, ld, max(lens), tree_mask=pack([mask], T).cuda(),
                                           k_scales=ks, v_scales=vs)
        return qr, out, lse

    qr, out, lse = step()
    k, v = fa.fa_cache_gather(kp, vp, td, ld, max(lens), dtype=torch.float32, k_scales=ks, v_scales=vs)
    rows = [[x[b, :, :n].double().cpu().transpose(0, 1) for b, n in enumerate(lens)] for x in (k, v)]
    want = ref.tree_attention(qr.cpu(), rows[0], rows[1], [T] * B, [mask] * B, D ** -0.5)
    ref.check_tree(out, lse, want, BF16, D, "over the cache as written")
    # the whole in 64 bits: the cache's values are off by up to 2^-4 each way, the scores with them
    kk, vv = [], []
    for b, c in enumerate(ctx):
        hk = ref.rotate(hist[0][b:b + 1, :, :c], torch.arange(c)[None], f)
        nk = ref.rotate(kv[0][b:b + 1], pos[b:b + 1], f)
        kk.append(torch.cat((hk, nk), 2)[0].transpose(0, 1))
        vv.append(torch.cat((hist[1][b, :, :c], kv[1][b]), 1).double().transpose(0, 1))
    o = ref.tree_attention(ref.rotate(q, pos, f), kk, vv, [T] * B, [mask] * B, D ** -0.5)[0]
    rel = (out.double().cpu() - o).norm() / o.norm()
    assert rel < 2 ** -4  # rms of the roundings is well under their bound
    again = step()
    assert torch.equal(again[1], out) and torch.equal(again[2], lse)


def test_graph_replay_and_two_streams():
    """A captured call replayed on new lengths and queries equals the eager one; calls on two
    streams with a workspace each do not disturb one another."""
    pr = Problem(1, 8, 1, 5, 128, 16, BF16, E4M3, [3000])
    (q, k, v, table, lens, L), kw = pr.gpu()
    mask = pack([random_tree(5, random.Random(5))], 5).cuda()
    fa.fa_tree_decode_paged(q, k, v, table, lens, L, tree_mask=mask, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fa.fa_tree_decode_paged(q, k, v, table, lens, L, tree_mask=mask, **kw)
    q.copy_(torch.randn_like(q))
    lens.fill_(2777)
    graph.replay()
    eager = fa.fa_tree_decode_paged(q, k, v, table, lens, L, tree_mask=mask, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    q2 = torch.randn_like(q)
    want2 = fa.fa_tree_decode_paged(q2, k, v, table, lens, L, tree_mask=mask, **kw)
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((fa.fa_tree_decode_paged(q, k, v, table, lens, L, tree_mask=mask, stream=s1, **kw),
                    fa.fa_tree_decode_paged(q2, k, v, table, lens, L, tree_mask=mask, stream=s2, **kw)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0], eager[0]) and torch.equal(b[0], want2[0])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,T", [(8, 1), (9, 1), (4, 2), (3, 3), (16, 1), (5, 3), (17, 1)])
def test_eight_rows_and_the_next(D, G, T):
    """Rows (query heads of a kv head times drafted tokens) around one and two tiles of eight,
    lengths around a slice, long enough for several slices a warp."""
    lens = [T, 33, 300, 16 + T]
    pr = Problem(len(lens), 2 * G, 2, T, D, 16, BF16, E4M3, lens, scales=(100, 140))
    masks = [random_tree(T, random.Random(G + b)) for b in range(len(lens))]
    args, kw = pr.gpu()
    for splits in (1, 2):
        out, lse = fa.fa_tree_decode_paged(*args, tree_mask=pack(masks, T).cuda(), num_splits=splits, **kw)
        ref.check_tree(out, lse, pr.want([T] * len(lens), masks, D ** -0.5), BF16, D, f"G={G} T={T} {splits}")


@pytest.mark.parametrize("D,G,T", [(128, 2, 3), (128, 4, 4), (64, 3, 5), (256, 4, 2), (256, 5, 3)])
def test_padding_queries_of_few_rows(D, G, T):
    """What the queries of padding rows hold (NaN, infinities, the largest values) changes no bit
    of the other rows, whose weights share their blocks' arithmetic."""
    pr = Problem(2, 2 * G, 2, T, D, 16, BF16, E4M3, [700, 77])
    (q, *rest), kw = pr.gpu()
    drafts = torch.tensor([1, T - 1], dtype=torch.int32, device="cuda")
    good = fa.fa_tree_decode_paged(q, *rest, draft_lens=drafts, num_splits=1, **kw)
    for bad in (math.nan, math.inf, 3e38, 0.0):
        q[0, :, 1:] = bad
        q[1, :, T - 1:] = bad
        out, lse = fa.fa_tree_decode_paged(q, *rest, draft_lens=drafts, num_splits=1, **kw)
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (FP16, FP16), (BF16, E4M3)])
@pytest.mark.parametrize("D,G,T,ps", [(128, 5, 1, 32), (128, 4, 2, 8), (64, 2, 1, 8), (256, 4, 1, 64), (128, 4, 9, 16), (64, 33, 1, 16)])
def test_short_sequences(dtype, cache, D, G, T, ps):
    """Lengths around every step of 16 tokens and a tile; NaN in every slot past a sequence's end
    and in pages that no sequence has."""
    lens = [n for n in (1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 128, 129, 145) if n >= T]
    pr = Problem(len(lens), 2 * G, 2, T, D, ps, dtype, cache, lens)
    used = torch.zeros(pr.k.shape[0], ps, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[pr.table[b, j // ps], j % ps] = True
    nan = 0x7f if cache == E4M3 else math.nan
    past = (~used)[:, None, :, None].expand(pr.k.shape)
    pr.k[past], pr.v[past] = nan, nan
    masks = [random_tree(T, random.Random(b)) for b in range(len(lens))]
    args, kw = pr.gpu()
    out, lse = fa.fa_tree_decode_paged(*args, tree_mask=pack(masks, T).cuda(), **kw)
    ref.check_tree(out, lse, pr.want([T] * len(lens), masks, D ** -0.5), dtype, D)
