"""The operators of a packed prompt, of its training step and of a recurrent decode step, as
measured workloads, each with its plain form in elementary torch operations:

* ``norm``: RMS norms of queries and keys for each head with the rotary positions in the same
  pass, and the gradient of both with respect to the inputs and the norms' weights;
* ``packed``: attention over whole prompts, sequences of different lengths behind one another in
  one tensor, grouped heads, causal (or not), keys that may reach further back than the queries;
  and its gradient;
* ``step``: the gated delta rule token by token, on a pool of states (one token: a decode step).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
GOLDEN = 0.6180339887498949
EPS = 1e-6


def listed():
    return [
        # five short prompts of one scheduler step; latency counts
        dict(name="packed_short_prompts", op="packed", B=5, len_min=1, len_max=64, extra=0, Hq=32,
             Hkv=8, D=128, dtype="bf16", causal=True, grad=False),
        # a prefill batch of prompts of 128 to 2048 tokens
        dict(name="packed_prompt_batch", op="packed", B=16, len_min=128, len_max=2048, extra=0,
             Hq=32, Hkv=8, D=128, dtype="bf16", causal=True, grad=False),
        # one user's long prompt
        dict(name="packed_long_prompt", op="packed", B=1, len_min=16384, len_max=16384, extra=0,
             Hq=16, Hkv=4, D=128, dtype="bf16", causal=True, grad=False),
        # chunked prefill: ragged chunks at the end of contexts, an odd group of heads
        dict(name="packed_chunks_fp16", op="packed", B=6, len_min=1, len_max=509, extra=6000,
             Hq=20, Hkv=4, D=64, dtype="fp16", causal=True, grad=False),
        # the gradient of a few short samples, one kv head a query head
        dict(name="packed_gradient_short", op="packed", B=3, len_min=37, len_max=200, extra=0,
             Hq=8, Hkv=8, D=64, dtype="fp16", causal=True, grad=True),
        # the gradient of a training batch packed from samples of 512 to 2048 tokens
        dict(name="packed_gradient_batch", op="packed", B=8, len_min=512, len_max=2048, extra=0,
             Hq=32, Hkv=8, D=128, dtype="bf16", causal=True, grad=True),
        # the gradient of one long sample
        dict(name="packed_gradient_long", op="packed", B=1, len_min=8192, len_max=8192, extra=0,
             Hq=16, Hkv=4, D=128, dtype="bf16", causal=True, grad=True),
        # a decode step of 128 sequences, one token each; latency counts
        dict(name="norm_decode_step", op="norm", B=128, T=1, Hq=32, Hk=8, D=128, rot=128,
             interleaved=False, dtype="bf16", weight="bf16", far=4096, grad=False),
        # a 16K-token prompt
        dict(name="norm_prompt", op="norm", B=1, T=16384, Hq=32, Hk=8, D=128, rot=128,
             interleaved=False, dtype="bf16", weight="bf16", far=131072, grad=False),
        # gradients in fp32, an odd length, half of each head rotated
        dict(name="norm_gradient", op="norm", B=2, T=1843, Hq=16, Hk=16, D=64, rot=32,
             interleaved=True, dtype="fp32", weight="fp32", far=8192, grad=True),
        # one token of each of 128 sequences through the recurrent layer
        dict(name="step_decode_batch", op="step", B=128, T=1, Hk=16, Hv=32, dtype="bf16",
             ragged=False),
        # one user's few drafted tokens, the state before them kept
        dict(name="step_one_user", op="step", B=1, T=5, Hk=16, Hv=32, dtype="bf16", ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "packed", "packed", "packed", "norm", "norm", "step", "step"])
    if op == "packed":
        grad = rng.random() < 0.5
        Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([64, 128])
        B = _log_int(rng, 1, 64)
        # what the scores of all heads, padded, may hold
        most = (400_000_000 if grad else 1_500_000_000) // (B * Hkv * G)
        hi = _log_int(rng, 1, max(2, min(8192, int(most ** 0.5))))
        extra = 0
        if not grad and rng.random() < 0.4:
            extra = min(8192, max(0, most // hi - hi))
            extra = _log_int(rng, 1, extra) if extra > 1 else 0
        return dict(op=op, B=B, len_min=rng.randrange(0, hi + 1), len_max=hi, extra=extra,
                    Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    causal=rng.random() < 0.8, grad=grad)
    if op == "norm":
        Hk, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 80, 128, 192, 256])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        grad = rng.random() < 0.5
        most = 16384 * 40 * 128 // (Hk * (G + 1) * D * (SIZE[dtype] // 2))
        tokens = min(_log_int(rng, 1, max(2, most)), 20000 if grad else 40000)
        B = min(tokens, _log_int(rng, 1, 64))
        return dict(op=op, B=B, T=max(1, tokens // B), Hq=Hk * G, Hk=Hk, D=D,
                    rot=rng.choice([D, D // 32 * 16]), interleaved=rng.random() < 0.5, dtype=dtype,
                    weight=rng.choice([dtype, "fp32"]), far=_log_int(rng, 2048, 1 << 20), grad=grad)
    Hk = rng.choice([1, 2, 4, 8, 16])
    B = _log_int(rng, 1, 128)
    return dict(op=op, B=B, T=rng.choice([1, 1, 2, 3, 5, 8]), Hk=Hk, Hv=Hk * rng.choice([1, 2]),
                dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.4)


def _spread(n, lo, hi, phase=0.5):
    """n lengths over lo..hi, the same for every seed (the work of a case is then known)."""
    return [lo + int((hi - lo) * ((i * GOLDEN + phase) % 1.0) + 0.5) for i in range(n)]


def _lens(case):
    """Queries and keys of each sequence."""
    q = _spread(case["B"], case["len_min"], case["len_max"])
    return q, [n + e for n, e in zip(q, _spread(case["B"], 0, case["extra"], 0.25))]


def _new_lens(case):
    return _spread(case["B"], 0, case["T"]) if case["ragged"] else [case["T"]] * case["B"]


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    op, dev, dt = case["op"], "cuda", DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "packed":
        ql, kl = _lens(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        s["max_q"], s["max_k"] = max(ql), max(kl)
        s["cu_q"] = torch.tensor(_offsets(ql), dtype=torch.int32, device=dev)
        s["cu_k"] = torch.tensor(_offsets(kl), dtype=torch.int32, device=dev) if case["extra"] else None
        # as the projection leaves them: one row a token, heads side by side (the keys of longer
        # contexts come from elsewhere)
        Tq, Tk = sum(ql), sum(kl)
        qkv = torch.randn((Tq, Hq + 2 * Hkv, D), generator=gen, device=dev, dtype=dt)
        s["q"] = qkv[:, :Hq]
        kv = qkv[:, Hq:]
        if case["extra"]:
            kv = torch.randn((Tk, 2 * Hkv, D), generator=gen, device=dev, dtype=dt)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        s["scale"] = 1.0 / math.sqrt(D)
        if case["grad"]:
            s["dout"] = torch.randn((Tq, Hq, D), generator=gen, device=dev, dtype=dt)
            # what the forward pass left
            s["out"], s["lse"] = _plain_packed(s)
        return s
    if op == "norm":
        B, T, D, Hq, Hk = case["B"], case["T"], case["D"], case["Hq"], case["Hk"]
        # heads and tokens differ in size, as projections do
        qk = torch.randn((B, T, Hq + Hk, D), generator=gen, device=dev, dtype=torch.float32)
        qk = (qk * torch.exp(torch.randn((B, T, Hq + Hk, 1), generator=gen, device=dev))).to(dt)
        s["q"], s["k"] = qk[:, :, :Hq].transpose(1, 2), qk[:, :, Hq:].transpose(1, 2)
        w = 1.0 + 0.2 * torch.randn((2, D), generator=gen, device=dev)
        w = w.to(DTYPES[case["weight"]])
        s["q_weight"], s["k_weight"] = w[0].clone(), w[1].clone()
        start = torch.randint(0, max(1, case["far"] - T + 1), (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = 10000.0 ** (-2.0 * i / case["rot"])
        if case["grad"]:
            s["dq_out"] = torch.randn((B, Hq, T, D), generator=gen, device=dev, dtype=dt)
            s["dk_out"] = torch.randn((B, Hk, T, D), generator=gen, device=dev, dtype=dt)
        return s
    B, T, Hk, Hv, D = case["B"], case["T"], case["Hk"], case["Hv"], 128
    x = torch.randn((B, T, Hk, 2 * D), generator=gen, device=dev, dtype=torch.float32)
    x = x / x.view(B, T, Hk, 2, D).norm(dim=-1, keepdim=True).expand(-1, -1, -1, -1, D).reshape(x.shape)
    x = x.to(dt)
    s["q"], s["k"] = x[..., :D].transpose(1, 2), x[..., D:].transpose(1, 2)
    s["v"] = torch.randn((B, T, Hv, D), generator=gen, device=dev, dtype=dt).transpose(1, 2)
    s["g"] = -0.005 - 0.245 * torch.rand((B, Hv, T), generator=gen, device=dev)
    s["beta"] = torch.rand((B, Hv, T), generator=gen, device=dev)
    # a pool of states in use; each sequence's state is read from one slot and written to another,
    # so that rejected drafts can be taken back
    slots = torch.randperm(2 * B + 1, generator=cpu)
    s["states"] = 0.3 * torch.randn((2 * B + 1, Hv, D, D), generator=gen, device=dev)
    s["read"] = slots[:B].to(dev, torch.int32)
    s["write"] = slots[B:2 * B].to(dev, torch.int32)
    s["new_lens"] = (torch.tensor(_new_lens(case), dtype=torch.int32, device=dev)
                     if case["ragged"] else None)
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# -------------------------------------------------------------------------------- plain forms
def _padded(x, cu, L):
    """Packed [total,H,D] as [B,H,L,D] in fp32, zeros behind each sequence."""
    t = torch.arange(L, device=x.device)
    rows = x[(cu[:-1, None] + t).clamp(max=x.shape[0] - 1).long()].float()
    inside = t < (cu[1:] - cu[:-1])[:, None]
    return torch.where(inside[..., None, None], rows, 0.0).transpose(1, 2)


def _packed(x, cu, total):
    """Padded [B,H,L,...] as [total,H,...]."""
    t = torch.arange(total, device=x.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return x[b, :, t - cu[b]]


def _scores(s):
    """Queries, keys and values, padded, and the scores [B,Hkv,G*Lq,Lk], -inf where nothing is seen."""
    case, Lq, Lk = s["case"], s["max_q"], s["max_k"]
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    cu_q, cu_k = s["cu_q"], s["cu_q"] if s["cu_k"] is None else s["cu_k"]
    q = _padded(s["q"], cu_q, Lq).reshape(B, Hkv, -1, D)
    k, v = _padded(s["k"], cu_k, Lk), _padded(s["v"], cu_k, Lk)
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None, None], (cu_k[1:] - cu_k[:-1])[:, None, None]
    i = torch.arange(Lq, device=q.device)[:, None]
    j = torch.arange(Lk, device=q.device)
    seen = (i < nq) & (j < nk)
    if case["causal"]:
        seen = seen & (j <= i + nk - nq)
    x = ((q * s["scale"]) @ k.transpose(2, 3)).view(B, Hkv, -1, Lq, Lk)
    x = x.masked_fill_(~seen[:, None, None], -math.inf).view(B, Hkv, -1, Lk)
    return q, k, v, x


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (x - m).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, total.log() + m


def _plain_packed(s):
    case, cu, total = s["case"], s["cu_q"], s["q"].shape[0]
    B, Hq, Lq, D = case["B"], case["Hq"], s["max_q"], case["D"]
    _, _, v, x = _scores(s)
    p, norm, lse = _softmax(x)
    out = torch.where(norm > 0, (p @ v) / norm, 0.0).view(B, Hq, Lq, D)
    return (_packed(out, cu, total).to(s["q"].dtype),
            _packed(lse.view(B, Hq, Lq), cu, total))


def _plain_packed_grad(s):
    case, cu_q = s["case"], s["cu_q"]
    cu_k = cu_q if s["cu_k"] is None else s["cu_k"]
    B, Hq, Hkv, D, Lq = case["B"], case["Hq"], case["Hkv"], case["D"], s["max_q"]
    dt = s["q"].dtype
    q, k, v, x = _scores(s)
    p, norm, _ = _softmax(x)
    p = torch.where(norm > 0, p / norm, 0.0)
    do = _padded(s["dout"], cu_q, Lq).reshape(B, Hkv, -1, D)
    dv = p.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
    dq = (ds @ k).view(B, Hq, Lq, D)
    dk = ds.transpose(2, 3) @ q
    Tk = s["k"].shape[0]
    return (_packed(dq, cu_q, s["q"].shape[0]).to(dt), _packed(dk, cu_k, Tk).to(dt),
            _packed(dv, cu_k, Tk).to(dt))


def _turned(x, s, back):
    """The first columns of x [B,H,T,D] turned by their angles (or back)."""
    half = s["inv_freq"].numel()
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    c, n = angle.cos().float(), angle.sin().float()
    if back:
        n = -n
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    inter = s["case"]["interleaved"]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :half], r[..., half:])
    ya, yb = a * c - b * n, b * c + a * n
    y = torch.stack((ya, yb), -1).flatten(-2) if inter else torch.cat((ya, yb), -1)
    return torch.cat((y, rest), -1)


def _plain_norm(x, w, s):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _turned(x * r * w.float(), s, False)


def _plain_norm_grad(dy, x, w, s):
    """Gradients of the input and, in fp32, of the weight."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    g = _turned(dy.float(), s, True)
    h = g * w.float()
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    # over heads and tokens: many values of either sign, in 64 bits
    return dx, (g * n).double().sum((0, 1, 2)).float()


def _plain_step(s):
    case, read, write = s["case"], s["read"].long(), s["write"].long()
    G = case["Hv"] // case["Hk"]
    q, k = (s[n].float().repeat_interleave(G, 1) for n in ("q", "k"))
    v, g, beta = s["v"].float(), s["g"], s["beta"]
    S = s["states"][read]
    out = torch.zeros_like(v)
    for t in range(case["T"]):  # a recurrence: each token needs the state that the last one left
        kt, qt, bt = k[:, :, t], q[:, :, t], beta[:, :, t, None]
        new = S * g[:, :, t].exp()[..., None, None]
        u = bt * (v[:, :, t] - (new @ kt[..., None])[..., 0])
        new = new + u[..., None] * kt[..., None, :]
        o = (new @ qt[..., None])[..., 0] * s["scale"]
        if s["new_lens"] is not None:
            live = (t < s["new_lens"])[:, None, None]
            new, o = torch.where(live[..., None], new, S), torch.where(live, o, 0.0)
        S = new
        out[:, :, t] = o
    s["states"][write] = S
    return out.to(s["q"].dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import softmax_attention_gb300 as fa
        if op == "packed" and case["grad"]:
            return fa.fa_prefill_packed_backward(s["dout"], s["q"], s["k"], s["v"], s["out"],
                                                 s["lse"], s["cu_q"], s["cu_k"],
                                                 causal=case["causal"], scale=s["scale"])
        if op == "packed":
            return fa.fa_prefill_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                        causal=case["causal"], scale=s["scale"])
        if op == "norm" and case["grad"]:
            return fa.fa_qk_norm_rotary_backward(s["dq_out"], s["dk_out"], s["q"], s["k"],
                                                 s["positions"], s["inv_freq"], s["q_weight"],
                                                 s["k_weight"], eps=EPS,
                                                 interleaved=case["interleaved"])
        if op == "norm":
            return fa.fa_qk_norm_rotary(s["q"], s["k"], s["positions"], s["inv_freq"],
                                        s["q_weight"], s["k_weight"], eps=EPS,
                                        interleaved=case["interleaved"])
        out = fa.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"],
                                  read_index=s["read"], write_index=s["write"],
                                  new_lens=s["new_lens"], scale=s["scale"])
        return out, s["states"]
    if op == "packed":
        return _plain_packed_grad(s) if case["grad"] else _plain_packed(s)
    if op == "norm" and case["grad"]:
        dq, wq = _plain_norm_grad(s["dq_out"], s["q"], s["q_weight"], s)
        dk, wk = _plain_norm_grad(s["dk_out"], s["k"], s["k_weight"], s)
        return dq.to(s["q"].dtype), dk.to(s["k"].dtype), wq, wk
    if op == "norm":
        return (_plain_norm(s["q"], s["q_weight"], s).to(s["q"].dtype),
                _plain_norm(s["k"], s["k_weight"], s).to(s["k"].dtype))
    return _plain_step(s), s["states"]


# ---------------------------------------------------------------------------------- 64 bits
def _exact_packed(case, s):
    """Sequence by sequence and kv head by kv head; the gradients by differentiation."""
    (ql, kl), Hq, Hkv, D = _lens(case), case["Hq"], case["Hkv"], case["D"]
    qo, ko = _offsets(ql), _offsets(kl)
    f64 = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros((qo[-1], Hq, D), **f64)
    lse = torch.full((qo[-1], Hq), -math.inf, **f64)
    dq, dk, dv = torch.zeros_like(out), torch.zeros((ko[-1], Hkv, D), **f64), torch.zeros((ko[-1], Hkv, D), **f64)
    G = Hq // Hkv
    for b in range(case["B"]):
        n, m = ql[b], kl[b]
        if n == 0 or m == 0:
            continue
        rows, keys = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1) if case["causal"] else None
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            q, k, v = s["q"][rows, heads].double(), s["k"][keys, h].double(), s["v"][keys, h].double()
            if case["grad"]:
                q, k, v = (x.requires_grad_() for x in (q, k, v))
            x = torch.einsum("igd,jd->gij", q, k) * s["scale"]
            if hidden is not None:
                x = x.masked_fill(hidden, -math.inf)
            o = torch.einsum("gij,jd->igd", torch.softmax(x, -1), v)
            if case["grad"]:
                dq[rows, heads], dk[keys, h], dv[keys, h] = torch.autograd.grad(
                    o, (q, k, v), s["dout"][rows, heads].double())
            else:
                out[rows, heads] = o
                lse[rows, heads] = torch.logsumexp(x, -1).T
    return (dq, dk, dv) if case["grad"] else (out, lse)


def _exact_norm(x, w, s):
    """Unit-norm rows, and complex numbers turned by their angles."""
    half = s["inv_freq"].numel()
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
    if half == 0:
        return y
    th = torch.einsum("bt,f->btf", s["positions"].double(), s["inv_freq"])
    turn = torch.polar(torch.ones_like(th), th)[:, None]
    z = y[..., :2 * half]
    z = z.unflatten(-1, (half, 2)) if s["case"]["interleaved"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    z = z if s["case"]["interleaved"] else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), y[..., 2 * half:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "packed":
        return _exact_packed(case, s)
    if case["op"] == "norm":
        got = []
        for x, w, dy in (("q", "q_weight", "dq_out"), ("k", "k_weight", "dk_out")):
            x, w = s[x].double(), s[w].double()
            if case["grad"]:
                x, w = x.requires_grad_(), w.requires_grad_()
                got.append(torch.autograd.grad(_exact_norm(x, w, s), (x, w), s[dy].double()))
            else:
                got.append(_exact_norm(x, w, s))
        if case["grad"]:
            return got[0][0], got[1][0], got[0][1], got[1][1]
        return tuple(got)
    G = case["Hv"] // case["Hk"]
    states = s["states"].double()
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    eye = torch.eye(128, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_new_lens(case)):
        S = states[int(s["read"][b])].clone()
        for t in range(n):
            k = s["k"][b, :, t].double().repeat_interleave(G, 0)
            beta = s["beta"][b, :, t].double()[:, None, None]
            S = s["g"][b, :, t].double().exp()[:, None, None] * torch.einsum(
                "hvk,hkl->hvl", S, eye - beta * torch.einsum("hk,hl->hkl", k, k))
            S = S + beta * torch.einsum("hv,hk->hvk", s["v"][b, :, t].double(), k)
            out[b, :, t] = torch.einsum("hvk,hk->hv", S, s["scale"]
                                        * s["q"][b, :, t].double().repeat_interleave(G, 0))
        states[int(s["write"][b])] = S
    return out, states


def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "packed":
        ql, kl = _lens(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        pairs = sum(n * (m - n) + n * (n + 1) // 2 if case["causal"] else n * m for n, m in zip(ql, kl))
        rows, keys = sum(ql) * Hq, 2 * sum(kl) * Hkv
        if case["grad"]:  # q, out, its gradient and dq; k, v and theirs
            return {"bytes": size * D * (4 * rows + 2 * keys) + 4 * rows, "flops": 10 * pairs * Hq * D}
        return {"bytes": size * D * (2 * rows + keys) + 4 * rows, "flops": 4 * pairs * Hq * D}
    if op == "norm":
        tokens = case["B"] * case["T"]
        rows = tokens * (case["Hq"] + case["Hk"])
        passes = 3 if case["grad"] else 2
        extra = 4 * tokens + 4 * case["rot"] + 2 * case["D"] * SIZE[case["weight"]]
        return {"bytes": passes * rows * case["D"] * size + extra + (8 * case["D"] if case["grad"] else 0),
                "flops": rows * (3 * case["rot"] + (9 if case["grad"] else 4) * case["D"])}
    lens, Hk, Hv, D = _new_lens(case), case["Hk"], case["Hv"], 128
    tokens = sum(lens)
    return {"bytes": 2 * case["B"] * Hv * D * D * 4 + tokens * (2 * (Hk + Hv) * D * size + 8 * Hv),
            "flops": tokens * Hv * 7 * D * D}
