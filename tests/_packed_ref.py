"""Plain 64-bit references of the packed-prompt operators, with bounds on how far a result held in
16 bits on the way may be from them.

u is half a step of the operands' type, relative (torch.finfo(t).eps / 2), and e = 2^-24 that of
fp32.  What the bounds count:
  scores   D products summed in fp32 (2 D e of sum |q k| scale, to allow for sums that truncate),
           and a handful of roundings of the exponent itself (8 e of |s| + |lse| + 1)
  weights  P rounded once to 16 bits (u); the sums of its products in fp32 (2 n e)
  dS       0 where a row sees one key (in dk, where the sequence has one); else e_p of the weight, dP's and delta's errors times the weight (delta's with
           out's rounding where a row sees more than 16 keys), one rounding to 16 bits (u,
           and in fp16 half the least subnormal over the power of two that it is held times)
  results  one rounding to 16 bits (u)
"""
import math

import torch

E = 2.0 ** -24


def spans(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _visible(n, m, causal):
    i, j = torch.arange(n)[:, None], torch.arange(m)
    return (j <= i + m - n) if causal else torch.ones(n, m, dtype=torch.bool)


def _power(top):
    """The power of two that brings top to [8, 16)."""
    return 2.0 ** (3 - math.floor(math.log2(top))) if top > 0 else 1.0


def attention(q, k, v, causal, scale, dout=None, call_top=None, in_place_of=None):
    """One sequence in fp64: q [n,Hq,D], k, v [m,Hkv,D].  Returns a dict of name -> (value, bound):
    out, lse and, with dout, dq, dk, dv."""
    t = q.dtype
    u = torch.finfo(t).eps / 2
    tiny = torch.finfo(t).tiny * torch.finfo(t).eps
    n, Hq, D = q.shape
    m, Hkv = k.shape[:2]
    G = Hq // Hkv
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    kk, vv = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    if m == 0:
        zero = torch.zeros(n, Hq, D, dtype=torch.float64)
        got = {"out": (zero, zero), "lse": (torch.full((n, Hq), -math.inf, dtype=torch.float64),
                                            torch.zeros(n, Hq, dtype=torch.float64))}
        if dout is not None:
            empty = torch.zeros(0, Hkv, D, dtype=torch.float64)
            got |= {"dq": (zero, zero), "dk": (empty, empty), "dv": (empty, empty)}
        return got
    seen = _visible(n, m, causal)
    s = (q @ kk.transpose(1, 2)) * scale
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(seen, (s - torch.where(lse == -math.inf, 0.0, lse)[..., None]).exp(), 0.0)
    mag = (q.abs() @ kk.abs().transpose(1, 2)) * abs(scale)
    finite = torch.where(lse == -math.inf, 0.0, lse)
    es = 2 * D * E * mag + 8 * E * (torch.where(seen, s, 0.0).abs() + finite.abs()[..., None] + 1)
    es = torch.where(seen, es, 0.0).amax(-1, keepdim=True)  # of a row's scores, and so of its lse
    out = p @ vv
    a = p @ vv.abs()
    e_out = (u + 2 * es + 2 * m * E) * a + (u + 2 * es) * out.abs() + tiny
    got = {"out": (out.transpose(0, 1), e_out.transpose(0, 1)),
           "lse": (lse.T, (es[..., 0] + 8 * E * (finite.abs() + 1)).T)}
    if dout is None:
        return got
    do = dout.double().transpose(0, 1)
    f_row = torch.tensor([[_power(x) for x in row] for row in do.abs().amax(-1).tolist()], dtype=torch.float64)
    f_call = _power(call_top if call_top is not None else do.abs().max().item())
    ep = 4 * es + 8 * E
    dp = do @ vv.transpose(1, 2)
    delta = (do * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    e_dp = 2 * D * E * (do.abs() @ vv.abs().transpose(1, 2))
    e_delta = (do.abs() * (e_out + 2 * D * E * out.abs())).sum(-1, keepdim=True)
    # of a row that sees 16 keys at most delta is sum p dp / sum p, without out's rounding: each weight off by ep, above
    # and below, and each dp by e_dp; 16 sums and a division
    e_few = (p * (e_dp + (2 * ep + 80 * E) * dp.abs())).sum(-1, keepdim=True)
    count = seen.sum(-1, keepdim=True)
    e_delta = torch.where(count <= 16, e_few, e_delta)
    half = t == torch.float16
    e_ds = (ep + u) * ds.abs() + p * (e_dp + e_delta) * (1 + u)
    hidden = torch.where(seen, 1.0, 0.0)
    e_q = e_ds + (hidden * (2.0 ** -25 / f_row)[..., None] if half else 0.0)
    e_k = e_ds + (hidden * (2.0 ** -25 / f_call) if half else 0.0)
    # the only key's weight is 1: no gradient (exactly none in dq, and in dk if it is the sequence's only one)
    ds, e_q = (torch.where(count == 1, 0.0, x) for x in (ds, e_q))
    e_k = torch.zeros_like(e_k) if m == 1 else e_k
    e_p = (ep + u) * p + (hidden * 2.0 ** -25 / 128 if half else 0.0)
    heads = lambda x: x.view(Hkv, G, m, D).sum(1)  # noqa: E731  (a kv head's query heads)
    dq = ds @ kk * scale
    b_dq = abs(scale) * (e_q @ kk.abs() + 2 * m * E * (ds.abs() @ kk.abs()))
    dk = heads(ds.transpose(1, 2) @ q) * scale
    b_dk = abs(scale) * heads(e_k.transpose(1, 2) @ q.abs() + 2 * G * n * E * (ds.abs().transpose(1, 2) @ q.abs()))
    dv = heads(p.transpose(1, 2) @ do)
    b_dv = heads(e_p.transpose(1, 2) @ do.abs() + 2 * G * n * E * (p.transpose(1, 2) @ do.abs()))
    for name, x, b in (("dq", dq, b_dq), ("dk", dk, b_dk), ("dv", dv, b_dv)):
        got[name] = (x.transpose(0, 1), (b * (1 + u) + u * x.abs() + tiny).transpose(0, 1))
    return got


def check(name, got, want, bound):
    """Within the bound; infinities equal."""
    got = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), f"{name}: infinities differ"
    off = (got[fine] - want[fine]).abs()
    bad = ~(off <= bound[fine])
    if bad.any():
        worst = (off / bound[fine].clamp(min=1e-300)).nan_to_num(math.inf).max().item()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values past their bound, "
                             f"the worst by {worst:.3g} times")
