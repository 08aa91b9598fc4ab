"""GPU checks of the norms of queries and keys with rotary positions, and of their gradient, against
plain 64-bit references."""
import math

import pytest
import torch

import softmax_attention_gb300 as fa
from tests import _cache_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def _freqs(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)


def _turn(x, pos, f, amp, il, back=False):
    return x if f is None else ref.rotate(x, pos, f, amp, il, back)


def _pairs(x, f, il):
    """|x_a| + |x_b| of each element's pair; |x| where nothing turns (the norm's error is in these
    columns as well)."""
    return x.abs() if f is None else ref.pair_sum(x, f, il).maximum(x.abs())


def _turn_error(x, pos, f, amp, il):
    """Of the rotation in fp32: 8 e of amp times the pair, and 2^-52 of the angle on either side."""
    if f is None:
        return torch.zeros_like(x)
    th = pos.double().abs().max() * f.max()
    return _pairs(x, f, il) * amp * (8 * E + 2 * 2.0 ** -52 * th)


def _round(dtype, x, slack):
    """One rounding to dtype on top of what fp32 may be off by."""
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    return (x.abs() + slack) * torch.finfo(dtype).eps / 2 + slack + tiny


def _norm(x, w, eps):
    r = (x.pow(2).mean(-1, keepdim=True) + eps) ** -0.5
    return r, x * r * w


def _inside(got, want, bound):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} past their bound"


CASES = [
    # B, Hq, Hk, T, D, rot, interleaved, dtype, weight type, first position, eps
    (1, 1, 1, 1, 16, 16, False, SF, SF, 3, 1e-6),
    (2, 4, 2, 5, 128, 128, False, BF, BF, 0, 1e-6),
    (2, 4, 2, 5, 128, 64, True, BF, SF, 1000, 1e-5),
    (1, 32, 8, 1, 128, 128, False, HF, HF, 131071, 1e-6),
    (1, 3, 1, 17, 80, 32, True, SF, SF, 12345, 1e-6),       # five units in eight lanes
    (3, 5, 5, 7, 64, 64, False, SF, SF, 1 << 20, 1e-6),
    (1, 2, 1, 33, 96, 96, False, BF, BF, 50, 1e-6),
    (2, 9, 0, 3, 256, 256, True, BF, BF, 4000, 1e-6),       # no keys
    (1, 64, 2, 2, 512, 512, False, BF, SF, 99, 1e-6),
    (1, 2, 2, 4, 192, 64, False, HF, SF, -20, 1e-3),        # negative positions
    (1, 3, 1, 6, 208, 0, False, BF, BF, 0, 1e-6),           # norms alone
    (1, 8, 8, 9, 32, 16, True, HF, HF, 7, 0.0),             # no epsilon
    (1, 40, 8, 700, 128, 128, False, BF, BF, 0, 1e-6),      # several heads a thread
    (2, 17, 3, 301, 64, 32, False, SF, SF, 5, 1e-6),
    (1, 3, 2, 5, 256, 128, True, SF, SF, 77, 1e-6),         # fp32: the widest rows in units of eight columns
    (1, 3, 2, 5, 272, 160, False, SF, SF, 77, 1e-6),        # and in units of sixteen
    (2, 2, 1, 3, 512, 512, True, SF, SF, 1 << 16, 1e-6),
    (1, 2, 3, 9, 16, 16, True, HF, HF, 11, 1e-6),           # a row a lane
]


class Case:
    def __init__(self, B, Hq, Hk, T, D, rot, il, dtype, wtype, first, eps, packed=True):
        g = torch.Generator().manual_seed(B + T + D + Hq)
        qk = torch.randn(B, T, Hq + Hk, D, generator=g) * torch.exp(torch.randn(B, T, Hq + Hk, 1, generator=g))
        qk = qk.to(dtype)
        dev = qk.cuda()
        cut = lambda x: (x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2))  # noqa: E731
        self.q, self.k = cut(qk)
        self.qd, self.kd = cut(dev) if packed else [x.contiguous() for x in cut(dev)]
        w = (1 + 0.3 * torch.randn(2, D, generator=g)).to(wtype)
        self.w = [w[0], w[1]]
        self.pos = (first + torch.arange(B * T, dtype=torch.int32)).view(B, T)
        self.f = _freqs(rot) if rot else None
        self.dy = torch.randn(B, T, Hq + Hk, D, generator=g).to(dtype)
        self.dqo, self.dko = cut(self.dy)
        self.dqod, self.dkod = cut(self.dy.cuda())
        self.dtype, self.il, self.eps, self.amp = dtype, il, eps, 1.25
        self.args = (self.pos.cuda(), self.f.cuda()) if rot else (None, None)
        self.kw = dict(eps=eps, amplitude=self.amp, interleaved=il)
        self.Hk = Hk
        self.on_gpu = None

    def keys(self, x):
        return x if self.Hk else None

    def weights(self):
        if self.on_gpu is None:
            self.on_gpu = [w.cuda() for w in self.w]
        return self.on_gpu

    def forward(self, **kw):
        return fa.fa_qk_norm_rotary(self.qd, self.keys(self.kd), *self.args, *self.weights(), **self.kw, **kw)

    def backward(self, **kw):
        return fa.fa_qk_norm_rotary_backward(self.dqod, self.keys(self.dkod), self.qd, self.keys(self.kd),
                                             *self.args, *self.weights(), **self.kw, **kw)

    def check_forward(self, got):
        for x, w, y in zip((self.q, self.k)[:2 if self.Hk else 1], self.w, got):
            _, n = _norm(x.double(), w.double(), self.eps)
            want = _turn(n, self.pos, self.f, self.amp, self.il)
            # the mean of squares sums D terms (D e at most), the root halves it; four more roundings
            slack = (x.shape[-1] / 2 + 4) * E * _pairs(n, self.f, self.il) * self.amp
            slack = slack + _turn_error(n, self.pos, self.f, self.amp, self.il)
            _inside(y, want, _round(self.dtype, want, slack))

    def check_backward(self, got):
        parts = ((self.q, self.dqo), (self.k, self.dko))[:2 if self.Hk else 1]
        for i, (x, dy) in enumerate(parts):
            x, dy, w = x.double(), dy.double(), self.w[i].double()
            D = x.shape[-1]
            r, _ = _norm(x, w, self.eps)
            n = x * r
            g = _turn(dy, self.pos, self.f, self.amp, self.il, True)
            eg = _turn_error(dy, self.pos, self.f, self.amp, self.il) + 2 * E * g.abs()
            mean = (g * w * n).mean(-1, keepdim=True)
            size = (g * w * n).abs().mean(-1, keepdim=True)
            want = r * (g * w - n * mean)
            # r is good to (D/2 + 4) e; the mean sums D terms more; a handful of products
            er = (D / 2 + 4) * E
            slack = r * (eg * w.abs() + n.abs() * (eg * w.abs() * n.abs()).mean(-1, keepdim=True)
                         + (3 * er + (D + 8) * E) * ((g * w).abs() + n.abs() * size))
            _inside(got[i], want, _round(self.dtype, want, slack))
            rows = x.numel() // D
            total = (g * n).sum((0, 1, 2))
            bound = (eg * n.abs()).sum((0, 1, 2)) + (er + (rows + 4) * E) * (g * n).abs().sum((0, 1, 2))
            _inside(got[2 + i], total, bound)


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, packed):
    c = Case(*case, packed=packed)
    c.check_forward(c.forward())


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    c = Case(*case)
    got = c.backward()
    c.check_backward(got)
    again = c.backward()
    for a, b in zip(got, again):  # no atomics
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("case", CASES[:5])
def test_in_place(case):
    c = Case(*case)
    want = c.forward()
    grad = c.backward()
    into = c.backward(dq=c.dqod, dk=c.keys(c.dkod))
    assert into[0].data_ptr() == c.dqod.data_ptr()
    for a, b in zip(grad, into):
        assert torch.equal(a, b)
    got = c.forward(q_out=c.qd, k_out=c.keys(c.kd))
    assert got[0].data_ptr() == c.qd.data_ptr()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_without_weights_and_keys():
    c = Case(2, 4, 2, 5, 128, 128, False, BF, BF, 0, 1e-6)
    c.w = [torch.ones(128, dtype=BF), torch.ones(128, dtype=BF)]
    want = c.forward()
    got = fa.fa_qk_norm_rotary(c.qd, c.kd, *c.args, None, None, **c.kw)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    grad = c.backward()
    dq, dk, wq, wk = fa.fa_qk_norm_rotary_backward(c.dqod, None, c.qd, None, *c.args, None, **c.kw)
    assert torch.equal(dq, grad[0]) and dk is None and wq is None and wk is None


def test_broadcast_inputs():
    """Heads that share one row's storage: strides of 0."""
    x = torch.randn(1, 1, 6, 64, device="cuda")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    f = _freqs(64).cuda()
    w = torch.rand(64, device="cuda")
    y, _ = fa.fa_qk_norm_rotary(x.expand(1, 8, 6, 64), None, pos, f, w)
    z, _ = fa.fa_qk_norm_rotary(x.repeat(1, 8, 1, 1), None, pos, f, w)
    assert torch.equal(y, z)


def test_captured_and_on_a_stream():
    c = Case(1, 8, 2, 33, 128, 128, False, BF, BF, 40, 1e-6)
    want, grad = c.forward(), c.backward()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for a, b in zip(want + grad, c.forward(stream=s) + c.backward(stream=s)):
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.forward() + c.backward()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want + grad, got):
            assert torch.equal(a, b)


def test_extreme_rows():
    """A row of zeros, one of the least numbers and one of large ones, in fp32."""
    x = torch.zeros(1, 1, 3, 64)
    x[0, 0, 1] = 1e-30
    x[0, 0, 2] = 1e15
    y, _ = fa.fa_qk_norm_rotary(x.cuda(), None, None, None, None)
    want = x.double() * (x.double().pow(2).mean(-1, keepdim=True) + 1e-6) ** -0.5
    torch.testing.assert_close(y.double().cpu(), want, rtol=1e-5, atol=1e-30)
    dy = torch.ones_like(x).cuda()
    dx, _, _, _ = fa.fa_qk_norm_rotary_backward(dy, None, x.cuda(), None, None, None, None)
    assert torch.isfinite(dx).all()
    torch.testing.assert_close(dx[0, 0, 0].cpu(), torch.full((64,), 1e3), rtol=1e-5, atol=0)


def test_gradient_against_differences():
    c = Case(1, 3, 2, 7, 64, 32, True, SF, SF, 11, 1e-6)
    got = c.backward()
    h = 1e-5
    gen = torch.Generator().manual_seed(1)

    def loss(q, k, wq, wk):
        total = 0.0
        for x, w, dy in ((q, wq, c.dqo), (k, wk, c.dko)):
            total += (_turn(_norm(x, w, c.eps)[1], c.pos, c.f, c.amp, c.il) * dy.double()).sum().item()
        return total

    inputs = [c.q.double(), c.k.double(), c.w[0].double(), c.w[1].double()]
    for i, grad in enumerate(got):
        d = torch.randn(inputs[i].shape, generator=gen, dtype=torch.float64)
        d = d * (inputs[i].norm() / d.norm()) if i < 2 else d
        up = [x + h * d if j == i else x for j, x in enumerate(inputs)]
        down = [x - h * d if j == i else x for j, x in enumerate(inputs)]
        slope = (loss(*up) - loss(*down)) / (2 * h)
        mine = (grad.double().cpu() * d).sum().item()
        assert math.isclose(mine, slope, rel_tol=1e-4, abs_tol=1e-4), (i, mine, slope)


def test_as_two_calls():
    """The same as the norm alone followed by fa_rotary, but for the rounding between."""
    c = Case(1, 8, 2, 50, 128, 128, False, SF, SF, 9, 1e-6)
    one = c.forward()
    q, k = fa.fa_qk_norm_rotary(c.qd, c.kd, None, None, *c.weights(), eps=c.eps)
    two = fa.fa_rotary(q, k, *c.args, amplitude=c.amp)
    for a, b in zip(one, two):
        torch.testing.assert_close(a, b, rtol=2e-6, atol=2e-6)
