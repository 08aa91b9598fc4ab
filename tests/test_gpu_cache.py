"""GPU checks of rotary positions and of the paged cache's write and read, against plain 64-bit
references (tests/_cache_ref.py).

What can be compared exactly is: an 8-bit row's codes and scale byte (the scale is a power of
two, so the one rounding is to e4m3), 16-bit copies, and everything read back.  A rotated value
carries the fp32 evaluation's error and one rounding to its type.
"""
import math

import pytest
import torch

import softmax_attention_gb300 as fa
from tests import _cache_ref as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def _freqs(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)


def _rotary_bound(x, want, positions, f, amp, interleaved, dtype):
    """Half a step of the output's type, and the fp32 evaluation: the phase reaches the sine as
    fp32 half turns (rounding 2^-25 of one, pi 2^-25 < 1.6 2^-24 rad), sine and cosine are good
    to 2 steps, then the amplitude, two products and a sum round: in all less than 8 * 2^-24 of
    amp (|x_a| + |x_b|).  The angle itself is a product in 64 bits on either side: 2^-52 of it
    each."""
    pair = ref.pair_sum(x, f, interleaved)
    th = positions.cpu().double().abs().max() * f.max()
    slack = pair * amp * (8 * 2.0 ** -24 + 2 * 2.0 ** -52 * th)
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # half a step among subnormals
    return want.abs() * torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -10) + slack + tiny


ROTARY = [
    # B, Hq, Hk, T, D, rot, interleaved, transpose, dtype, first position
    (2, 4, 2, 5, 128, 128, False, False, torch.bfloat16, 0),
    (2, 4, 2, 5, 128, 128, True, False, torch.bfloat16, 1000),
    (1, 32, 8, 1, 128, 64, False, False, torch.float16, 131071),
    (1, 3, 1, 17, 80, 32, True, True, torch.float32, 12345),
    (3, 5, 5, 7, 64, 64, False, True, torch.float32, 1 << 20),
    (1, 1, 1, 1, 16, 16, False, False, torch.float32, 7),
    (1, 2, 1, 33, 72, 64, False, False, torch.bfloat16, 50),     # a trailing unit of eight columns
    (1, 2, 1, 9, 24, 16, True, False, torch.float16, 50),
    (2, 9, 0, 3, 256, 256, True, False, torch.bfloat16, 4000),   # no keys
    (1, 64, 2, 2, 512, 512, False, False, torch.bfloat16, 99),
    (1, 2, 2, 4, 192, 64, False, True, torch.float16, -20),      # negative positions
    (1, 40, 8, 700, 128, 128, False, False, torch.bfloat16, 0),  # several heads a thread
]


@pytest.mark.parametrize("B,Hq,Hk,T,D,rot,il,tr,dtype,first", ROTARY)
@pytest.mark.parametrize("packed", [True, False])
def test_rotary(B, Hq, Hk, T, D, rot, il, tr, dtype, first, packed):
    g = torch.Generator().manual_seed(B + T + D)
    qk = torch.randn(B, T, Hq + Hk, D, generator=g).to(dtype)
    q, k = qk[:, :, :Hq].transpose(1, 2), qk[:, :, Hq:].transpose(1, 2)
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    pos = (first + torch.arange(B * T, dtype=torch.int32)).view(B, T)
    f, amp = _freqs(rot), 1.25
    if packed:
        dev = qk.cuda()
        qd, kd = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:].transpose(1, 2)
    else:
        qd, kd = q.cuda(), k.cuda()
    oq, ok = fa.fa_rotary(qd, kd if Hk else None, pos.cuda(), f.cuda(), amplitude=amp,
                          interleaved=il, transpose=tr)
    for x, y in ((q, oq), (k, ok)) if Hk else ((q, oq),):
        want = ref.rotate(x, pos, f, amp, il, tr)
        err = (y.double().cpu() - want).abs()
        assert (err <= _rotary_bound(x, want, pos, f, amp, il, dtype)).all(), err.max()
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
    # in place gives the same bits
    fa.fa_rotary(qd, kd if Hk else None, pos.cuda(), f.cuda(), amplitude=amp, interleaved=il,
                 transpose=tr, q_out=qd, k_out=kd if Hk else None)
    assert torch.equal(qd, oq) and (not Hk or torch.equal(kd, ok))


def test_rotary_far_positions():
    """Angles at the ends of int32: each position's phase is a 64-bit product, checked against
    exact rational arithmetic on quarter turns (f = pi/2 2^-k: position p turns p / 2^(k+2))."""
    k = torch.arange(8, dtype=torch.float64)
    f = math.pi / 2 * 2.0 ** -k
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 31 - 5, 123456789]], dtype=torch.int32)
    x = torch.zeros(1, 1, 4, 16)
    x[..., :8] = 1.0
    y, _ = fa.fa_rotary(x.cuda(), None, pos.cuda(), f.cuda())
    y = y.cpu().double()[0, 0]
    for i, p in enumerate(pos[0].tolist()):
        for j in range(8):
            den = 2 ** (j + 2)
            th = 2 * math.pi * (p % den) / den
            # f is pi/2 2^-k rounded (2^-53 of it): at 2^31 that is 2^-22 turns at most
            assert abs(y[i, j] - math.cos(th)) < 2.0 ** -19
            assert abs(y[i, 8 + j] - math.sin(th)) < 2.0 ** -19


def test_rotary_gradient():
    """transpose=True is the gradient: against the formula's in 64 bits (above) and against
    differences of a linear loss, which have no truncation error."""
    g = torch.Generator().manual_seed(3)
    q, w, d = (torch.randn(2, 3, 11, 64, generator=g) for _ in range(3))
    pos = torch.randint(0, 5000, (2, 11), generator=g, dtype=torch.int32).cuda()
    f = _freqs(48).cuda()

    def loss(x):
        return (fa.fa_rotary(x.cuda(), None, pos, f, amplitude=1.1)[0].double().cpu() * w).sum()

    grad, _ = fa.fa_rotary(w.cuda(), None, pos, f, amplitude=1.1, transpose=True)
    want = (loss(q + d) - loss(q - d)) / 2
    got = (grad.double().cpu() * d).sum()
    # 4224 products of O(1) on each side, each off by under 16 * 2^-24 of its size
    scale = (w.abs() * (q.abs() + d.abs())).sum().double()
    assert abs(want - got) <= 2 * 16 * 2.0 ** -24 * scale


def _pools(P, Hkv, ps, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if dtype == E4M3:
        codes = torch.randint(0, 0x7F, (2, P, Hkv, ps, D), generator=g, dtype=torch.uint8)
        codes += 128 * torch.randint(0, 2, codes.shape, generator=g, dtype=torch.uint8)
        scales = torch.randint(100, 150, (2, P, Hkv, ps), generator=g, dtype=torch.uint8)
        return codes[0], codes[1], scales[0], scales[1]
    x = torch.randn(2, P, Hkv, ps, D, generator=g).to(dtype)
    return x[0], x[1], None, None


def _on_gpu(pages, scales):
    if scales is None:
        return pages.cuda(), None
    return pages.cuda().view(E4M3), scales.cuda()


def _codes(pages):
    return pages.view(torch.uint8).cpu()


APPEND = [
    # B, T, Hkv, D, page, dtype, cache, lens (the new tokens included), new lens or None
    (2, 5, 2, 128, 16, torch.bfloat16, E4M3, [5, 40], None),
    (3, 7, 1, 64, 8, torch.float16, E4M3, [7, 9, 100], [7, 0, 3]),
    (1, 1, 8, 256, 64, torch.float32, E4M3, [1], None),
    (2, 33, 3, 128, 1, torch.bfloat16, E4M3, [40, 33], [33, 1]),      # one-token pages
    (2, 5, 2, 128, 16, torch.bfloat16, torch.bfloat16, [5, 40], [5, 2]),
    (1, 130, 5, 64, 32, torch.float16, torch.float16, [131], None),
    (5, 1, 4, 256, 128, torch.bfloat16, E4M3, [300, 1, 128, 129, 2], [1, 1, 0, 1, 1]),
]


@pytest.mark.parametrize("B,T,Hkv,D,ps,dtype,cache,lens,new", APPEND)
def test_append(B, T, Hkv, D, ps, dtype, cache, lens, new):
    g = torch.Generator().manual_seed(D + T)
    P = sum(-(-n // ps) for n in lens) + 3
    table = ref.make_table(lens, ps, P, g)
    kp, vp, ks, vs = _pools(P, Hkv, ps, D, cache, 11)
    kv = torch.randn(B, T, 2 * Hkv, D, generator=g) * torch.exp(3 * torch.randn(B, T, 2 * Hkv, 1, generator=g))
    kv = kv.to(dtype)
    dev = kv.cuda()
    k, v = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
    kd, vd = dev[:, :, :Hkv].transpose(1, 2), dev[:, :, Hkv:].transpose(1, 2)
    (kpd, ksd), (vpd, vsd) = _on_gpu(kp, ks), _on_gpu(vp, vs)
    nd = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    fa.fa_cache_append(kd, vd, kpd, vpd, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                       new_lens=nd, k_scales=ksd, v_scales=vsd)
    for x, pages, scales in ((k, kp, ks), (v, vp, vs)):
        for b in range(B):
            n = T if new is None else new[b]
            for t in range(n):
                pos = lens[b] - n + t
                page, slot = int(table[b, pos // ps]), pos % ps
                if cache == E4M3:
                    pages[page, :, slot], scales[page, :, slot] = ref.quantise(x[b, :, t])
                else:
                    pages[page, :, slot] = x[b, :, t]
    # the whole pools: the new slots as they should be, every other one as it was
    if cache == E4M3:
        assert torch.equal(_codes(kpd), kp) and torch.equal(_codes(vpd), vp)
        assert torch.equal(ksd.cpu(), ks) and torch.equal(vsd.cpu(), vs)
    else:
        assert torch.equal(kpd.cpu(), kp) and torch.equal(vpd.cpu(), vp)


def test_append_borders():
    """Rows at the borders of the scale and of e4m3: the largest value 448 2^k exactly and one
    fp32 step above, midpoints between e4m3 values, subnormal results, zeros, subnormal and huge
    rows, infinities and NaN."""
    rows = []
    for k in (-40, -3, 0, 5, 100):
        for m in (1.75, math.nextafter(1.75, 2.0), 1.0, 1.9999):
            r = torch.zeros(64)
            r[0] = math.ldexp(m, k)
            r[1:] = torch.linspace(-1, 1, 63) * r[0]
            rows.append(r)
            r = torch.zeros(64)
            r[0] = math.ldexp(1.75, k)
            r[1:34] = torch.tensor([math.ldexp(1 + (i + 0.5) / 8, k - 2 * (i % 8)) for i in range(33)])
            r[34:] = torch.tensor([math.ldexp(i / 2.0, k - 17) for i in range(30)])
            rows.append(r)
    rows.append(torch.zeros(64))
    rows.append(-torch.zeros(64))
    rows.append(torch.full((64,), 1e-42))
    rows.append(torch.linspace(-3.4e38, 3.4e38, 64))
    bad = torch.linspace(-5, 5, 64)
    bad[3], bad[7], bad[9] = math.inf, -math.inf, math.nan
    rows += [bad, torch.full((64,), math.inf), torch.full((64,), math.nan)]
    x = torch.stack(rows)[None, None].float()  # [1,1,T,64]
    T = x.shape[2]
    kp = torch.zeros(T, 1, 1, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    vp = kp.clone()
    ks = torch.zeros(T, 1, 1, dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    table = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    fa.fa_cache_append(x.cuda(), (-x).cuda(), kp, vp, table, lens, k_scales=ks, v_scales=vs)
    for sign, pages, scales in ((1, kp, ks), (-1, vp, vs)):
        codes, e = ref.quantise(sign * x[0, 0])
        got = _codes(pages)[:, 0, 0]
        nan = torch.isnan(x[0, 0])
        assert torch.equal(scales.cpu()[:, 0, 0], e)
        assert torch.equal(got[~nan], codes[~nan])
        assert ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("cache", [E4M3, torch.bfloat16])
@pytest.mark.parametrize("rot,given,T", [(128, True, 6), (64, False, 6), (32, False, 400)])
def test_append_rotated(il, cache, rot, given, T):
    """Keys rotated as they are written: once in fp32, rounded once."""
    g = torch.Generator().manual_seed(rot)
    B, Hkv, D, ps, lens = 2, 9, 128, 16, [T + 4, T + 27]
    P = sum(-(-n // ps) for n in lens) + 1
    table = ref.make_table(lens, ps, P, g)
    kp, vp, ks, vs = _pools(P, Hkv, ps, D, cache, 5)
    (kpd, ksd), (vpd, vsd) = _on_gpu(kp, ks), _on_gpu(vp, vs)
    k = torch.randn(B, Hkv, T, D, generator=g).to(torch.bfloat16)
    v = torch.randn(B, Hkv, T, D, generator=g).to(torch.bfloat16)
    pos = torch.stack([torch.arange(n - T, n, dtype=torch.int32) for n in lens])
    if given:
        pos = torch.randint(0, 100000, (B, T), generator=g, dtype=torch.int32)
    f, amp = _freqs(rot), 0.75
    fa.fa_cache_append(k.cuda(), v.cuda(), kpd, vpd, table.cuda(),
                       torch.tensor(lens, dtype=torch.int32).cuda(), k_scales=ksd, v_scales=vsd,
                       inv_freq=f.cuda(), amplitude=amp, interleaved=il,
                       positions=pos.cuda() if given else None)
    want = ref.rotate(k, pos, f, amp, il)
    bound = _rotary_bound(k, want, pos, f, amp, il, torch.float32)
    for b, n in enumerate(lens):
        rows = ref.rows_of(kpd.view(torch.uint8).cpu() if cache == E4M3 else kpd.cpu(), table, b, n)[n - T:]
        w, bd = want[b].transpose(0, 1), bound[b].transpose(0, 1)
        if cache == E4M3:
            sc = ref.rows_of(ksd.cpu(), table, b, n)[n - T:]
            got = ref.dequantise(rows, sc)
            amax = w.abs().amax(-1)
            e = sc.double() - 127
            # the scale is the least that holds the largest value, up to the fp32 error of it
            assert (amax <= 448 * 2 ** e * (1 + 1e-5)).all()
            assert (amax * (1 + 1e-5) >= 448 * 2 ** (e - 1)).all()
            # half a step of e4m3 (2^-4 of the value), or of its subnormals (2^-10 scales)
            lim = torch.maximum(w.abs() * 2.0 ** -4, 2.0 ** (e - 10)[..., None])
            assert ((got - w).abs() <= lim * (1 + 1e-5) + 2 * bd).all()
        else:
            assert ((rows.double() - w).abs() <= w.abs() * 2.0 ** -8 + bd).all()
    # values are not rotated
    for b, n in enumerate(lens):
        x = v[b].transpose(0, 1)
        if cache == E4M3:
            codes, e = ref.quantise(x)
            assert torch.equal(ref.rows_of(_codes(vpd), table, b, n)[n - T:], codes)
        else:
            assert torch.equal(ref.rows_of(vpd.cpu(), table, b, n)[n - T:], x)


GATHER = [
    # Hkv, D, page, cache, out, lens, max_len
    (2, 128, 16, E4M3, torch.bfloat16, [5, 40, 0], 40),
    (1, 64, 8, E4M3, torch.float16, [100], 103),
    (3, 256, 64, E4M3, torch.float32, [1, 129], 129),
    (2, 128, 1, torch.bfloat16, torch.bfloat16, [33, 7], 50),
    (2, 64, 32, torch.float16, torch.float32, [33, 64], 64),
    (8, 128, 128, torch.bfloat16, torch.float16, [700], 700),
]


@pytest.mark.parametrize("Hkv,D,ps,cache,out,lens,L", GATHER)
def test_gather(Hkv, D, ps, cache, out, lens, L):
    g = torch.Generator().manual_seed(L)
    P = sum(-(-n // ps) for n in lens) + 3
    table = ref.make_table(lens, ps, P, g, spare=60)
    kp, vp, ks, vs = _pools(P, Hkv, ps, D, cache, 7)
    (kpd, ksd), (vpd, vsd) = _on_gpu(kp, ks), _on_gpu(vp, vs)
    k, v = fa.fa_cache_gather(kpd, vpd, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                              L, dtype=out, k_scales=ksd, v_scales=vsd)
    for got, pages, scales in ((k, kp, ks), (v, vp, vs)):
        want = torch.zeros(len(lens), Hkv, L, D, dtype=torch.float64)
        for b, n in enumerate(lens):
            rows = ref.rows_of(pages, table, b, n)
            if cache == E4M3:
                rows = ref.dequantise(rows, ref.rows_of(scales, table, b, n))
            want[b, :, :n] = rows.double().transpose(0, 1)
        assert torch.equal(got.cpu(), want.to(out))  # one rounding: exact


def test_write_then_read():
    """Chunks appended one after another, read back whole: each value within half a step."""
    g = torch.Generator().manual_seed(2)
    B, Hkv, D, ps = 2, 2, 128, 16
    T, steps = 13, 4
    total = T * steps
    P = B * -(-total // ps)
    table = ref.make_table([total] * B, ps, P, g).cuda()
    kp = torch.zeros(P, Hkv, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    vp = kp.clone()
    ks = torch.zeros(P, Hkv, ps, dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    x = torch.randn(2, B, Hkv, total, D, generator=g).to(torch.bfloat16).cuda()
    for i in range(steps):
        lens = torch.full((B,), T * (i + 1), dtype=torch.int32, device="cuda")
        fa.fa_cache_append(x[0, :, :, i * T:(i + 1) * T], x[1, :, :, i * T:(i + 1) * T], kp, vp, table,
                           lens, k_scales=ks, v_scales=vs)
    got = fa.fa_cache_gather(kp, vp, table, lens, total, dtype=torch.float32, k_scales=ks, v_scales=vs)
    for y, w in zip(got, x):
        w = w.double()
        amax = w.abs().amax(-1, keepdim=True)
        # half a step: 2^-4 of the value, or 2^-10 of the scale, which is under 2 amax / 448
        assert ((y.double() - w).abs() <= torch.maximum(w.abs() * 2.0 ** -4, amax / 224 * 2.0 ** -10)).all()


def test_bad_pages_and_lengths_are_skipped():
    B, T, Hkv, D, ps, P = 4, 2, 1, 64, 8, 4
    pages = torch.zeros(P, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 99], [-1, 1], [2, 2], [3, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([9, 2, 1, 17], dtype=torch.int32, device="cuda")  # 1 < T; 17 > 2 pages
    vp = pages.clone()
    fa.fa_cache_append(k, k, pages, vp, table, lens)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    want = torch.zeros_like(pages)
    want[0, :, 7] = 1  # sequence 0's first new token (position 7); its second needs page 99
    assert torch.equal(pages, want) and torch.equal(vp, want)
    kk, _ = fa.fa_cache_gather(pages, vp, table, torch.tensor([8, 3, -1, 30], dtype=torch.int32).cuda(), 16)
    assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
    assert torch.equal(kk[0, 0, :8], want[0, 0]) and not kk[1:].any() and not kk[0, 0, 8:].any()


def test_side_stream_and_graph():
    """A step captured into a graph and replayed on new contents, and a call on a side stream."""
    B, T, Hkv, D, ps = 2, 1, 4, 128, 16
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    kp = torch.zeros(4, Hkv, ps, D, dtype=torch.uint8, device="cuda").view(E4M3)
    vp = kp.clone()
    ks = torch.zeros(4, Hkv, ps, dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    lens = torch.tensor([3, 17], dtype=torch.int32, device="cuda")
    pos = lens[:, None] - 1
    x = torch.randn(B, 2 * Hkv, T, D, device="cuda").to(torch.bfloat16)
    f = _freqs(64).cuda()

    def step():
        _, k = fa.fa_rotary(x[:, :Hkv], x[:, :Hkv], pos, f)
        fa.fa_cache_append(k, x[:, Hkv:], kp, vp, table, lens, k_scales=ks, v_scales=vs)
        return fa.fa_cache_gather(kp, vp, table, lens, 20, k_scales=ks, v_scales=vs)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(torch.randn_like(x))
    lens += 1
    pos.copy_(lens[:, None] - 1)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in got]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = fa.fa_cache_gather(kp, vp, table, lens, 20, k_scales=ks, v_scales=vs, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, again))
    eager = step()
    assert all(torch.equal(a, b) for a, b in zip(replayed, eager))
    assert replayed[0][0, :, 3].any() and replayed[0][1, :, 17].any()
