"""GPU checks of the gated delta rule token by token, against the recurrence in 64 bits with a bound
that follows the fp32 evaluation's error through it."""
import pytest
import torch

import softmax_attention_gb300 as fa

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def _inputs(B, T, Hk, Hv, dtype, slots, seed=0):
    g = torch.Generator().manual_seed(seed)
    qk = torch.randn(B, T, 2 * Hk, 128, generator=g)
    qk = (qk / qk.norm(dim=-1, keepdim=True)).to(dtype)
    v = torch.randn(B, T, Hv, 128, generator=g).to(dtype).transpose(1, 2)
    gate = -0.3 * torch.rand(B, T, Hv, generator=g).transpose(1, 2)
    beta = torch.rand(B, T, Hv, generator=g).transpose(1, 2)
    states = torch.randn(slots, Hv, 128, 128, generator=g)
    return qk[:, :, :Hk].transpose(1, 2), qk[:, :, Hk:].transpose(1, 2), v, gate, beta, states


def _reference(q, k, v, g, beta, S, n, scale):
    """One sequence: outputs and state with their bounds.  e_S: what the fp32 state may be off by.
    A dot product of 128 terms, 16 in a row and three levels, rounds 19 times; expf is good to two
    steps."""
    T, Hv = v.shape[1], v.shape[0]
    G = Hv // q.shape[0]
    dtype = v.dtype
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    out, e_out = torch.zeros(Hv, T, 128, dtype=torch.float64), torch.zeros(Hv, T, 128, dtype=torch.float64)
    e_S = torch.zeros_like(S)
    for t in range(n):
        kt, qt = (x[:, t].repeat_interleave(G, 0)[:, None] for x in (k, q))
        a, b = g[:, t].exp()[:, None], beta[:, t][:, None]
        sk, mag = (S * kt).sum(-1), (S * kt).abs().sum(-1)
        e_sk = (e_S * kt.abs()).sum(-1) + 19 * E * mag
        u = b * (v[:, t] - a * sk)
        e_u = b * (a * e_sk + 6 * E * (v[:, t].abs() + a * mag))
        sq = (S * qt).sum(-1)
        kq = (kt * qt).sum(-1)
        e_o = a * ((e_S * qt.abs()).sum(-1) + 25 * E * (S * qt).abs().sum(-1)) + e_u * kq.abs() + 25 * E * u.abs() * (kt * qt).abs().sum(-1)
        old = a[..., None] * S
        S = old + u[..., None] * kt
        e_S = a[..., None] * e_S + e_u[..., None] * kt.abs() + 5 * E * (old.abs() + (u[..., None] * kt).abs())
        o = (S * qt).sum(-1) * scale
        out[:, t] = o
        half = torch.finfo(dtype).eps / 2
        e_out[:, t] = scale * e_o * (1 + half) + (half + 2 * E) * o.abs() + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    return out, e_out, S, e_S + E * S.abs()


def _inside(got, want, bound):
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} past their bound"


CASES = [
    # B, T, Hk, Hv, dtype, separate slots, ragged
    (1, 1, 1, 1, BF, False, False),
    (3, 1, 2, 4, BF, True, False),
    (2, 7, 2, 2, HF, False, True),
    (40, 1, 4, 8, BF, False, False),     # a whole state a block
    (40, 3, 4, 8, HF, True, True),
    (1, 64, 1, 3, BF, True, False),
    (2, 0, 1, 1, BF, True, False),       # no token: the states are copied
]


@pytest.mark.parametrize("B,T,Hk,Hv,dtype,apart,ragged", CASES)
def test_step(B, T, Hk, Hv, dtype, apart, ragged):
    slots = 2 * B + 1
    q, k, v, g, beta, states = _inputs(B, T, Hk, Hv, dtype, slots, seed=B + T)
    perm = torch.randperm(slots, generator=torch.Generator().manual_seed(1))
    read, write = perm[:B], perm[B:2 * B] if apart else perm[:B]
    lens = [(5 * b + 3) % (T + 1) for b in range(B)] if ragged else [T] * B
    pool = states.cuda()
    out = torch.full((B, T, Hv, 128), 7.0, dtype=dtype, device="cuda").transpose(1, 2)
    got = fa.gated_delta_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), pool,
                              read_index=read.to("cuda", torch.int32),
                              write_index=write.to("cuda", torch.int32) if apart else None,
                              new_lens=torch.tensor(lens, dtype=torch.int32, device="cuda") if ragged else None,
                              scale=0.1, out=out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    want = states.double()
    bound = torch.zeros_like(want)
    for b in range(B):
        o, e_o, S, e_S = _reference(q[b], k[b], v[b], g[b], beta[b], states[read[b]], lens[b], 0.1)
        _inside(out[b], o, e_o)
        assert not out[b, :, lens[b]:].any()
        want[write[b]], bound[write[b]] = S, e_S
    _inside(pool, want, bound)  # all other slots as they were, bit for bit


def test_defaults():
    """Slots 0..B-1 in place, scale 1/sqrt(128)."""
    q, k, v, g, beta, states = _inputs(2, 2, 1, 2, BF, 3)
    pool = states.cuda()
    out = fa.gated_delta_step(*(x.cuda() for x in (q, k, v, g, beta)), pool)
    for b in range(2):
        o, e_o, S, e_S = _reference(q[b], k[b], v[b], g[b], beta[b], states[b], 2, 128 ** -0.5)
        _inside(out[b], o, e_o)
        _inside(pool[b], S, e_S)
    assert torch.equal(pool[2].cpu(), states[2])


def test_one_by_one_is_the_same():
    """Tokens in one call or a call each: the same bits; and a captured step, replayed."""
    q, k, v, g, beta, states = (x.cuda() for x in _inputs(3, 4, 2, 4, BF, 3, seed=5))
    a, b = states.clone(), states.clone()
    whole = fa.gated_delta_step(q, k, v, g, beta, a)
    parts = [fa.gated_delta_step(*(x[:, :, t:t + 1] for x in (q, k, v, g, beta)), b) for t in range(4)]
    assert torch.equal(whole, torch.cat(parts, 2)) and torch.equal(a, b)
    c = states.clone()
    bufs = [x[:, :, :1].clone() for x in (q, k, v, g, beta)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.gated_delta_step(*bufs, c)
    c.copy_(states)
    for t in range(4):
        for buf, x in zip(bufs, (q, k, v, g, beta)):
            buf.copy_(x[:, :, t:t + 1])
        graph.replay()
        assert torch.equal(out, whole[:, :, t:t + 1])
    assert torch.equal(c, a)


def test_continues_a_prefill():
    """Chunked prefill of a prompt, then steps: the recurrence over all of it.  (The prefill's own
    tolerance: 2 % of the largest value, in bf16 products.)"""
    B, L, T, Hk, Hv = 2, 150, 5, 2, 4
    q, k, v, g, beta, _ = _inputs(B, L + T, Hk, Hv, BF, 1, seed=9)
    dev = [x.cuda() for x in (q, k, v, g, beta)]
    head = [x[:, :, :L].contiguous() for x in dev]
    _, states = fa.gated_delta_prefill(*head)
    out = fa.gated_delta_step(*(x[:, :, L:] for x in dev), states)
    zero = torch.zeros(Hv, 128, 128)
    for b in range(B):
        o, _, S, _ = _reference(q[b], k[b], v[b], g[b], beta[b], zero, L + T, 128 ** -0.5)
        for got, want in ((out[b], o[:, L:]), (states[b], S)):
            assert (got.double().cpu() - want).abs().max() <= 2e-2 * want.abs().max()


def test_a_shared_state_is_read_twice():
    """Two sequences from one slot (a shared prompt), each to its own."""
    q, k, v, g, beta, states = _inputs(2, 1, 1, 1, BF, 3, seed=11)
    pool = states.cuda()
    idx = lambda *i: torch.tensor(i, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.gated_delta_step(*(x.cuda() for x in (q, k, v, g, beta)), pool, read_index=idx(1, 1), write_index=idx(0, 2))
    for b, slot in ((0, 0), (1, 2)):
        _, _, S, e_S = _reference(q[b], k[b], v[b], g[b], beta[b], states[1], 1, 128 ** -0.5)
        _inside(pool[slot], S, e_S)
    assert torch.equal(pool[1].cpu(), states[1])


def test_out_of_range_is_reported():
    q, k, v, g, beta, states = (x.cuda() for x in _inputs(3, 2, 1, 1, BF, 3, seed=12))
    idx = lambda *i: torch.tensor(i, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw in (dict(read_index=idx(0, 3, -1)), dict(write_index=idx(0, 7, -1)), dict(new_lens=idx(2, 3, -1))):
        pool = states.clone()
        out = fa.gated_delta_step(q, k, v, g, beta, pool, **kw)
        assert fa.fa_get_device_status() == fa.FA_ERR_BOUNDS
        assert out[0].any() and not out[1:].any()
        assert torch.equal(pool[1:], states[1:]) and not torch.equal(pool[0], states[0])
