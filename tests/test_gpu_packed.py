"""GPU checks of attention over packed prompts and of its gradient, against plain 64-bit references
with derived bounds (tests/_packed_ref.py)."""
import math

import pytest
import torch

import softmax_attention_gb300 as fa
from tests import _packed_ref as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


class Case:
    """Packed tensors on the CPU and the GPU: q's sequences start at row `first` and `behind` rows
    follow them; these rows, in all inputs, hold NaN.  With separate key lengths k and v stand alone,
    else q, k and v are slices of one projection."""

    def __init__(self, lens, Hq, Hkv, D, dtype, *, klens=None, first=0, behind=0, size=1.0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.klens = list(lens), list(klens if klens is not None else lens)
        self.cu = ref.spans(self.lens, first)
        self.cuk = self.cu if klens is None else ref.spans(self.klens)
        self.D, self.Hq, self.Hkv = D, Hq, Hkv
        self.dtype = dtype
        total = self.cu[-1] + behind
        x = torch.randn(total, Hq + 2 * Hkv, D, generator=g)
        x[:first] = NAN
        x[self.cu[-1]:] = NAN
        self.x = x.to(dtype)
        self.y = None if klens is None else torch.randn(max(1, self.cuk[-1]), 2 * Hkv, D, generator=g).to(dtype)
        do = torch.randn(total, Hq, D, generator=g) * size
        do[:first] = NAN
        do[self.cu[-1]:] = NAN
        self.do = do.to(dtype)

    def views(self, x, y):
        q = x[:, :self.Hq]
        kv = x[:, self.Hq:] if y is None else y[:self.cuk[-1]]
        return q, kv[:, :self.Hkv], kv[:, self.Hkv:]

    def cpu(self):
        return self.views(self.x, self.y)

    def gpu(self):
        return self.views(self.x.cuda(), None if self.y is None else self.y.cuda())

    def offsets(self):
        cu = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        return cu, None if self.y is None else torch.tensor(self.cuk, dtype=torch.int32, device="cuda")

    def want(self, causal, scale, grad=False):
        q, k, v = self.cpu()
        top = max([self.do[a:b].abs().max().item() for a, b in zip(self.cu, self.cu[1:]) if b > a] or [0.0])
        for b in range(len(self.lens)):
            rows, keys = slice(self.cu[b], self.cu[b + 1]), slice(self.cuk[b], self.cuk[b + 1])
            if rows.start == rows.stop:
                if grad and keys.start < keys.stop:
                    zero = torch.zeros(keys.stop - keys.start, self.Hkv, self.D, dtype=torch.float64)
                    yield rows, keys, {"dk": (zero, zero), "dv": (zero, zero)}
                continue
            yield rows, keys, ref.attention(q[rows], k[keys], v[keys], causal, scale,
                                            self.do[rows] if grad else None, top)


CASES = [
    # query lengths, key lengths (None: the same), Hq, Hkv, D, dtype, causal
    ([1], None, 1, 1, 64, BF, True),
    ([1], None, 8, 2, 128, HF, True),
    ([2, 0, 1, 3], None, 4, 4, 128, BF, True),
    ([127, 128, 129], None, 2, 2, 64, BF, True),
    ([31, 32, 33, 64, 65], None, 8, 2, 128, BF, True),
    ([300, 5, 0, 257], None, 6, 2, 128, BF, True),          # groups of three: unused rows in a tile
    ([300, 5, 0, 257], None, 6, 2, 64, HF, True),
    ([130, 77], None, 10, 2, 128, HF, False),               # groups of five
    ([130, 77], None, 10, 2, 64, BF, False),
    ([513, 200], None, 16, 1, 128, BF, True),               # groups of sixteen
    ([9, 40], None, 100, 1, 64, BF, True),                  # one token a tile
    ([3, 2], None, 128, 1, 128, HF, True),
    ([700], None, 4, 2, 128, BF, True),
    ([700], None, 4, 2, 64, BF, False),
    ([5, 60, 1, 0, 33], [300, 60, 129, 7, 1000], 8, 2, 128, BF, True),   # the end of longer contexts
    ([5, 60, 1, 0, 33], [300, 60, 129, 7, 1000], 8, 2, 64, HF, False),
    ([40, 200, 3], [10, 0, 3], 4, 2, 128, BF, True),        # rows in front of every key
    ([40, 200, 3], [10, 0, 3], 4, 4, 64, HF, True),
    ([1] * 40, None, 4, 1, 64, BF, True),                   # more than a warp of sequences
    ([3, 140, 0] * 50, None, 2, 1, 64, BF, True),           # more than find their place by level
    # several work items a block, one after another, ragged, with and without tiles that only half
    # of a pair of query tiles sees
    ([(37 * i) % 401 for i in range(24)], None, 8, 8, 64, BF, True),
    ([(53 * i) % 401 for i in range(24)], None, 8, 8, 128, HF, True),
    ([(61 * i) % 331 for i in range(20)], None, 24, 8, 128, BF, False),
    ([(71 * i) % 211 for i in range(30)], [(29 * i) % 307 for i in range(30)], 24, 8, 64, HF, True),
    ([(41 * i) % 211 for i in range(30)], [(83 * i) % 307 for i in range(30)], 24, 8, 128, BF, True),
    ([200, 1, 77] * 60, None, 4, 2, 128, BF, True),         # and past what find their place by level
]


@pytest.mark.parametrize("lens,klens,Hq,Hkv,D,dtype,causal", CASES)
def test_forward(lens, klens, Hq, Hkv, D, dtype, causal):
    c = Case(lens, Hq, Hkv, D, dtype, klens=klens, first=0 if klens else 3, behind=5, seed=D + Hq)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    out = torch.full((q.shape[0], Hq + 1, D), 7.0, dtype=dtype, device="cuda")[:, :Hq]  # strided
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    fa.fa_prefill_packed(q, k, v, *c.offsets(), causal=causal, scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    for rows, _, want in c.want(causal, scale):
        ref.check("out", out[rows], *want["out"])
        ref.check("lse", lse[rows], *want["lse"])
    for t in (out, lse):  # rows of no sequence
        assert (t[:c.cu[0]] == 7).all() and (t[c.cu[-1]:] == 7).all()


@pytest.mark.parametrize("splits", [2, 3, 11, 32])
@pytest.mark.parametrize("lens,klens,Hq,Hkv,D,dtype,causal", CASES)
def test_forward_split(lens, klens, Hq, Hkv, D, dtype, causal, splits):
    """Keys in parts: the same bounds (parts are joined in 32 bits); rows of no sequence as they were."""
    c = Case(lens, Hq, Hkv, D, dtype, klens=klens, first=0 if klens else 3, behind=5, seed=D + Hq)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    out = torch.full((q.shape[0], Hq + 1, D), 7.0, dtype=dtype, device="cuda")[:, :Hq]  # strided
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.full((32 * q.shape[0] * Hq * (D + 1) * 4 + 512,), 255, dtype=torch.uint8, device="cuda")  # NaN
    fa.fa_prefill_packed(q, k, v, *c.offsets(), causal=causal, scale=scale, out=out, lse=lse,
                         num_splits=splits, workspace=ws)
    torch.cuda.synchronize()
    for rows, _, want in c.want(causal, scale):
        ref.check("out", out[rows], *want["out"])
        ref.check("lse", lse[rows], *want["lse"])
    outside = torch.ones(q.shape[0], dtype=torch.bool)
    outside[c.cu[0]:c.cu[-1]] = False
    assert (out[outside.cuda()] == 7).all() and (lse[outside.cuda()] == 7).all()


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
def test_forward_split_by_rule(D, dtype):
    """A few tokens at the end of long contexts: the library's own choice of parts."""
    c = Case([1, 70, 0, 33], 8, 2, D, dtype, klens=[9000, 7001, 300, 4096], seed=3)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale)
    one, _ = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale, num_splits=1)
    torch.cuda.synchronize()
    for rows, _, want in c.want(True, scale):
        ref.check("out", out[rows], *want["out"])
        ref.check("lse", lse[rows], *want["lse"])
        ref.check("out", one[rows], *want["out"])


def test_split_captured_and_replayed():
    """A captured call whose workspace is the graph's own, replayed with other values."""
    c = Case([5, 60], 8, 2, 128, BF, klens=[3000, 2500], seed=4)
    d = Case([5, 60], 8, 2, 128, BF, klens=[3000, 2500], seed=5)
    scale = 1.0 / math.sqrt(128)
    q, k, v = (t.contiguous() for t in c.gpu())
    offsets = c.offsets()
    fa.fa_prefill_packed(q, k, v, *offsets, scale=scale, num_splits=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fa.fa_prefill_packed(q, k, v, *offsets, scale=scale, num_splits=5)
    for case in (c, d):
        for to, src in zip((q, k, v), case.gpu()):
            to.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for rows, _, want in case.want(True, scale):
            ref.check("out", out[rows], *want["out"])
            ref.check("lse", lse[rows], *want["lse"])


@pytest.mark.parametrize("lens,klens,Hq,Hkv,D,dtype,causal", CASES)
def test_backward(lens, klens, Hq, Hkv, D, dtype, causal):
    c = Case(lens, Hq, Hkv, D, dtype, klens=klens, first=0 if klens else 3, behind=5, seed=D + Hq)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), causal=causal, scale=scale)
    dq = torch.full((q.shape[0], Hq + 1, D), 7.0, dtype=dtype, device="cuda")[:, :Hq]
    dkv = torch.full((k.shape[0], 2 * Hkv, D), 7.0, dtype=dtype, device="cuda")
    dk, dv = dkv[:, :Hkv], dkv[:, Hkv:]
    fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), causal=causal,
                                  scale=scale, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    for rows, keys, want in c.want(causal, scale, grad=True):
        if "dq" in want:
            ref.check("dq", dq[rows], *want["dq"])
        ref.check("dv", dv[keys], *want["dv"])
        ref.check("dk", dk[keys], *want["dk"])
    for t, cu in ((dq, c.cu), (dk, c.cuk), (dv, c.cuk)):
        assert (t[:cu[0]] == 7).all() and (t[cu[-1]:] == 7).all()


@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** 10])
@pytest.mark.parametrize("D", [64, 128])
def test_backward_half_range(size, D):
    """fp16 gradients far below and far above 1 keep their bits."""
    c = Case([150, 20], 4, 2, D, HF, size=size, seed=3)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale)
    dq, dk, dv = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), scale=scale)
    for rows, keys, want in c.want(True, scale, grad=True):
        ref.check("dq", dq[rows], *want["dq"])
        ref.check("dk", dk[keys], *want["dk"])
        ref.check("dv", dv[keys], *want["dv"])


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scales(scale):
    """A negative scale, none, and one that makes scores of a hundred."""
    c = Case([200, 33], 4, 2, 128, BF, seed=4)
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale)
    dq, dk, dv = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), scale=scale)
    for rows, keys, want in c.want(True, scale, grad=True):
        for name, got in (("out", out[rows]), ("lse", lse[rows]), ("dq", dq[rows]), ("dk", dk[keys]), ("dv", dv[keys])):
            ref.check(name, got, *want[name])


def test_rising_scores():
    """Scores that rise from tile to tile, by less and by more than what is let stand."""
    for step in (0.02, 0.2):
        D, L = 64, 900
        c = Case([L], 2, 1, D, BF, seed=6)
        c.x[:, :2] = 0
        c.x[:, :2, 0] = 8.0
        c.x[:, 2, 0] = (torch.arange(L) * step).to(BF)
        q, k, v = c.gpu()
        out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=1.0)
        for rows, _, want in c.want(True, 1.0):
            ref.check("out", out[rows], *want["out"])
            ref.check("lse", lse[rows], *want["lse"])


def test_other_sequences_take_no_part():
    """NaN and infinities in every other sequence, and a sequence of NaN keys beside a clean one."""
    lens = [33, 100, 7, 129]
    c = Case(lens, 4, 2, 128, BF, seed=8)
    for b in (0, 2):
        c.x[c.cu[b]:c.cu[b + 1]] = NAN if b else math.inf
        c.do[c.cu[b]:c.cu[b + 1]] = NAN
    scale = 0.1
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale)
    dq, dk, dv = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), scale=scale)
    clean = Case(lens, 4, 2, 128, BF, seed=8)
    for b, (rows, keys, want) in enumerate(clean.want(True, scale, grad=True)):
        if b in (1, 3):
            for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
                ref.check(name, got[rows], *want[name])


def test_half_gradient_of_other_sequences_infinite():
    """fp16: dout of one sequence at the type's end; the other's gradients stay finite and, where the
    power of two leaves them bits, right."""
    c = Case([64, 64], 2, 2, 64, HF, seed=9)
    c.do[:64] = 65504.0
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=0.125)
    got = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), scale=0.125)
    for b, (rows, keys, want) in enumerate(c.want(True, 0.125, grad=True)):
        if b == 1:
            for name, t in zip(("dq", "dk", "dv"), got):
                ref.check(name, t[rows], *want[name])


def test_matches_the_dense_call():
    """One sequence is fa_prefill's problem."""
    c = Case([520], 8, 2, 128, BF, seed=11)
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=0.09)
    dense = [x.transpose(0, 1)[None].contiguous() for x in (q, k, v)]
    o2, l2 = fa.fa_prefill(*dense, causal=True, scale=0.09)
    torch.testing.assert_close(out, o2[0].transpose(0, 1), rtol=2 ** -7, atol=2 ** -8)
    torch.testing.assert_close(lse, l2[0].T, rtol=0, atol=1e-5)


def test_same_bits_twice_and_on_streams():
    """Repeated, on another stream, and with two calls in flight at once."""
    c = Case([300, 40, 513], 8, 2, 128, BF, seed=12)
    q, k, v = c.gpu()
    do = c.do.cuda()
    cu, _ = c.offsets()
    out, lse = fa.fa_prefill_packed(q, k, v, cu)
    first = (out, lse) + fa.fa_prefill_packed_backward(do, q, k, v, out, lse, cu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams * 2:
        o, m = fa.fa_prefill_packed(q, k, v, cu, stream=s)
        got.append((o, m) + fa.fa_prefill_packed_backward(do, q, k, v, o, m, cu, stream=s))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(first, g):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_captured_and_replayed(dtype):
    """One capture, replayed on other values and other lengths of the same total."""
    a = Case([100, 50, 20], 4, 2, 64, dtype, seed=13)
    b = Case([1, 169], 4, 2, 64, dtype, seed=14)
    x, do = a.x.cuda(), a.do.cuda()
    cu = torch.tensor(a.cu, dtype=torch.int32, device="cuda")
    q, k, v = a.views(x, None)

    def step():
        out, lse = fa.fa_prefill_packed(q, k, v, cu, scale=0.1)
        return (out, lse) + fa.fa_prefill_packed_backward(do, q, k, v, out, lse, cu, scale=0.1)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for case, offsets in ((a, a.cu), (b, b.cu + [170])):  # the same number of sequences
        x.copy_(case.x)
        do.copy_(case.do)
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for rows, keys, want in case.want(True, 0.1, grad=True):
            for name, t in zip(("out", "lse", "dq", "dk", "dv"), got):
                ref.check(name, t[rows], *want[name])


def test_against_differences():
    """The gradients along random directions are the differences of the 64-bit forward pass."""
    c = Case([90, 41], 4, 2, 64, HF, seed=15)
    scale, h = 0.125, 1e-4
    q, k, v = c.gpu()
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), scale=scale)
    grads = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *c.offsets(), scale=scale)

    def loss(q, k, v):
        total = 0.0
        for a, b in zip(c.cu, c.cu[1:]):
            x = torch.einsum("igd,jgd->gij", q[a:b], k[a:b].repeat_interleave(2, 1)) * scale
            x = x.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), -math.inf)
            o = torch.einsum("gij,jgd->igd", torch.softmax(x, -1), v[a:b].repeat_interleave(2, 1))
            total += (o * c.do[a:b].double()).sum().item()
        return total

    inputs = [x.double() for x in c.cpu()]
    g = torch.Generator().manual_seed(16)
    for i, grad in enumerate(grads):
        d = torch.randn(inputs[i].shape, generator=g, dtype=torch.float64)
        up = [x + h * d if j == i else x for j, x in enumerate(inputs)]
        down = [x - h * d if j == i else x for j, x in enumerate(inputs)]
        slope = (loss(*up) - loss(*down)) / (2 * h)
        mine = (grad.double().cpu() * d).sum().item()
        # a sum of N values of about the same size, each good to a few of fp16's steps
        size = grad.double().norm().item()
        assert abs(mine - slope) <= 8 * 2.0 ** -11 * size + 1e-6 * abs(slope) + 1e-4, (i, mine, slope)


def test_broken_offsets_are_reported():
    """Offsets that fall, or reach out of the tensor, make empty sequences."""
    c = Case([64, 64], 2, 2, 64, BF, seed=17)
    q, k, v = c.gpu()
    for offsets in ([0, 64, 32], [-5, 64, 128], [0, 64, 129], [0, 2 ** 31 - 1, 128]):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        out, lse = fa.fa_prefill_packed(q, k, v, cu)
        assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
        fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, torch.zeros_like(out), torch.zeros_like(lse), cu)
        assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert fa.fa_get_device_status() == fa.FA_OK


@pytest.mark.parametrize("lens,klens,Hq,Hkv,D,dtype,causal", [
    ([1, 1, 1], None, 4, 2, 64, BF, True),                   # one key each: dq and dk are 0
    ([1, 2, 3, 4, 5, 8], None, 6, 2, 128, BF, True),
    ([1, 2, 3, 4, 5, 8], None, 10, 2, 64, HF, True),
    ([15, 16, 17, 31, 32, 33, 70], None, 8, 2, 128, HF, True),       # either side of what few means, and of twice it
    ([31, 32, 33, 200], [15, 16, 17, 16], 8, 2, 64, BF, False),
    ([300, 40], [1, 1], 4, 1, 128, BF, False),               # many queries of one key
    ([90, 64], [40, 3], 12, 4, 64, BF, True),                # queries in front of every key, then the first of one
    ([90, 64], [40, 3], 3, 3, 128, HF, True),
    ([5, 40], None, 128, 1, 64, BF, True),                   # more rows of few keys than a block takes
    ([1000], [13], 16, 1, 128, HF, False),
])
def test_rows_of_few_keys(lens, klens, Hq, Hkv, D, dtype, causal):
    """Where dP and delta nearly cancel: bounds without the rounding of out, and zeros that are zeros."""
    c = Case(lens, Hq, Hkv, D, dtype, klens=klens, first=0 if klens else 3, behind=5, seed=31 + D + Hq)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    offsets = c.offsets()
    out, lse = fa.fa_prefill_packed(q, k, v, *offsets, causal=causal, scale=scale)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # NaN
    dq, dk, dv = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, *offsets, causal=causal,
                                               scale=scale, workspace=ws)
    torch.cuda.synchronize()
    for rows, keys, want in c.want(causal, scale, grad=True):
        for name, got, at in (("dq", dq, rows), ("dk", dk, keys), ("dv", dv, keys)):
            if name in want:
                ref.check(name, got[at], *want[name])
    if lens == [1, 1, 1]:
        assert not dq[c.cu[0]:c.cu[-1]].any() and not dk[c.cu[0]:c.cu[-1]].any()


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
def test_many_sequences(D, dtype):
    """Seven hundred short samples: every block goes through many of them."""
    c = Case([(13 * i) % 17 for i in range(700)], 4, 2, D, dtype, first=2, behind=3, seed=21)
    scale = 1.0 / math.sqrt(D)
    q, k, v = c.gpu()
    cu, _ = c.offsets()
    out, lse = fa.fa_prefill_packed(q, k, v, cu, scale=scale)
    dq, dk, dv = fa.fa_prefill_packed_backward(c.do.cuda(), q, k, v, out, lse, cu, scale=scale)
    torch.cuda.synchronize()
    got = {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    for rows, _, want in c.want(True, scale, grad=True):
        for name, (value, bound) in want.items():
            ref.check(name, got[name][rows], value, bound)


def test_broken_offsets_with_parts():
    """Rows of a sequence that is taken as empty stay as they were, whatever the workspace holds."""
    c = Case([64, 64], 2, 2, 64, BF, seed=17)
    q, k, v = c.gpu()
    for offsets, first, end in (([0, 64, 32], 0, 64), ([-5, 64, 128], 64, 128), ([0, 64, 129], 0, 64),
                                ([0, 2 ** 31 - 1, 128], 0, 0)):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        out = torch.full((128, 2, 64), 7.0, dtype=BF, device="cuda")
        lse = torch.full((128, 2), 7.0, device="cuda")
        ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")  # NaN
        fa.fa_prefill_packed(q, k, v, cu, num_splits=2, out=out, lse=lse, workspace=ws)
        assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
        left = torch.ones(128, dtype=torch.bool, device="cuda")
        left[first:end] = False
        assert (out[left] == 7).all() and (lse[left] == 7).all()
        assert not (out[first:end] == 7).all() if end > first else True
        assert out.isfinite().all() and lse.isfinite().all()
    assert fa.fa_get_device_status() == fa.FA_OK


def test_parts_on_two_streams_at_once():
    """Two calls that overlap, a workspace each: the bits of the same calls alone."""
    cases = [Case([40, 7], 8, 2, 128, BF, klens=[6000, 3000], seed=s) for s in (6, 7)]
    ins = [(*c.gpu(), *c.offsets()) for c in cases]
    alone = [fa.fa_prefill_packed(*x, num_splits=6) for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(3):
        got = [fa.fa_prefill_packed(*x, num_splits=6, stream=s) for x, s in zip(ins, streams)]
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(alone, got):
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_parts_and_causal_rows_in_front():
    """Infinite scores and NaN in keys that a row's part does not see take no part."""
    c = Case([300], 4, 2, 64, HF, klens=[900], seed=8)
    q, k, v = c.gpu()
    k, v = k.clone(), v.clone()
    k[700:] = float("inf")  # seen by the rows from 100 on alone
    out, lse = fa.fa_prefill_packed(q, k, v, *c.offsets(), num_splits=7)
    one, lone = fa.fa_prefill_packed(q, k, v, *c.offsets(), num_splits=1)
    torch.cuda.synchronize()
    ref_rows = next(c.want(True, 1.0 / 8.0))[2]
    for got, l in ((out, lse), (one, lone)):
        ref.check("out", got[:100], *(t[:100] for t in ref_rows["out"]))
        ref.check("lse", l[:100], *(t[:100] for t in ref_rows["lse"]))


def test_no_rows():
    empty = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = fa.fa_prefill_packed(empty, empty[:, :2], empty[:, :2], cu)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # keys of a sequence without queries get zeros
    kv = torch.randn(5, 2, 64, device="cuda").to(BF)
    cuk = torch.tensor([0, 5, 5], dtype=torch.int32, device="cuda")
    dq, dk, dv = fa.fa_prefill_packed_backward(empty, empty, kv, kv, empty, lse, cu, cuk)
    assert dq.shape == (0, 4, 64) and not dk.any() and not dv.any()
    one = cu[:1]
    fa.fa_prefill_packed(kv, kv, kv, one)  # no sequence at all
    torch.cuda.synchronize()


def test_long_sequences():
    """Thousands of tokens: the forward pass against the dense call, the gradients by what holds for
    any size: dv sums to dout's sum where every row sees a key (weights sum to 1), and <dq, q> and <dk, k>
    to the same number."""
    lens = [4100, 1, 2000, 6001]
    c = Case(lens, 8, 2, 128, BF, seed=21)
    q, k, v = c.gpu()
    cu, _ = c.offsets()
    out, lse = fa.fa_prefill_packed(q, k, v, cu)
    do = c.do.cuda()
    dq, dk, dv = fa.fa_prefill_packed_backward(do, q, k, v, out, lse, cu)
    u = 2.0 ** -8
    for a, b in zip(c.cu, c.cu[1:]):
        dense = [x[a:b].transpose(0, 1)[None].contiguous() for x in (q, k, v)]
        o2, l2 = fa.fa_prefill(*dense, causal=True)
        # both round weights and results once: u each, of values of at most 1 in the mean
        torch.testing.assert_close(out[a:b].float(), o2[0].transpose(0, 1).float(), rtol=2 * u, atol=2 * u)
        torch.testing.assert_close(lse[a:b], l2[0].T, rtol=1e-6, atol=2e-5)
        n = b - a
        heads = lambda t: t[a:b].double().view(n, 2, -1, 128).sum((0, 2))  # noqa: E731
        # n * 4 terms of size about 1, each good to a few u at random: 6 standard deviations
        off = (dv[a:b].double().sum(0) - heads(do)).abs().max().item()
        assert off <= 6 * 2 * u * (4 * n) ** 0.5, off
        x, y = (dq[a:b].double() * q[a:b].double()).sum().item(), (dk[a:b].double() * k[a:b].double()).sum().item()
        size = (dq[a:b].double() * q[a:b].double()).norm().item() + (dk[a:b].double() * k[a:b].double()).norm().item()
        assert abs(x - y) <= 6 * 2 * u * size, (x, y, size)


def test_large_offsets():
    """Rows past 2^31 elements into the tensors."""
    H, D, L = 64, 128, 200
    first = (1 << 31) // (3 * H * D) + 1000
    x = torch.empty(first + L, 3 * H, D, dtype=BF, device="cuda")
    x[first:] = torch.randn(L, 3 * H, D, device="cuda").to(BF)
    q, k, v = x[:, :H], x[:, H:2 * H], x[:, 2 * H:]
    cu = torch.tensor([first, first + L], dtype=torch.int32, device="cuda")
    out, lse = fa.fa_prefill_packed(q, k, v, cu)
    small = x[first:]
    o2, l2 = fa.fa_prefill_packed(small[:, :H], small[:, H:2 * H], small[:, 2 * H:], cu - first)
    assert torch.equal(out[first:], o2) and torch.equal(lse[first:], l2)
    do = torch.empty_like(out)
    do[first:] = 1.0
    got = fa.fa_prefill_packed_backward(do, q, k, v, out, lse, cu)
    want = fa.fa_prefill_packed_backward(do[first:], small[:, :H], small[:, H:2 * H], small[:, 2 * H:], o2, l2, cu - first)
    for a, b in zip(got, want):
        assert torch.equal(a[first:], b)
