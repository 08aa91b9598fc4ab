"""The serving-step operators around the paged cache, as measured workloads.

Four operators, each with its plain form in elementary torch operations:

* ``rotary``: rotary positions on the queries and keys of a step (and their transpose, which is
  the gradient);
* ``append``: writing a step's keys and values into a paged cache, in 8 bits (e4m3 values and one
  power-of-two scale a token and head) or in the inputs' 16 bits with the rotation fused in;
* ``gather``: reading a paged cache back as dense keys and values;
* ``tree``: attention of a tree of drafted tokens over a paged cache (one token: plain decode).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
GOLDEN = 0.6180339887498949


def listed():
    return [
        # a decode step of 128 sequences: one token each, grouped heads; latency counts
        dict(name="rotary_decode_step", op="rotary", B=128, T=1, Hq=32, Hk=8, D=128, rot=128,
             interleaved=False, transpose=False, dtype="bf16", scaling="none", far=4096),
        # a 16K-token prompt at positions scaled to a long context, half of each head rotated
        dict(name="rotary_prompt_scaled", op="rotary", B=1, T=16384, Hq=32, Hk=8, D=128, rot=64,
             interleaved=True, transpose=False, dtype="bf16", scaling="by_parts", far=131072),
        # gradients of queries and keys in fp32, an odd length
        dict(name="rotary_gradient", op="rotary", B=2, T=1843, Hq=16, Hk=16, D=64, rot=64,
             interleaved=False, transpose=True, dtype="fp32", scaling="linear", far=8192),
        # the cache write of a decode step of 128 sequences, quantised
        dict(name="append_decode_q8", op="append", B=128, T=1, Hkv=8, D=128, page=16, dtype="bf16",
             cache="e4m3", rot=0, interleaved=False, len_min=1024, len_max=4096, ragged=False),
        # the cache write of 512-token chunks of 8 sequences (chunked prefill), quantised
        dict(name="append_chunk_q8", op="append", B=8, T=512, Hkv=8, D=128, page=16, dtype="bf16",
             cache="e4m3", rot=0, interleaved=False, len_min=2048, len_max=8192, ragged=False),
        # a padded batch of short prompts into a 16-bit cache, keys rotated as they are written
        dict(name="append_ragged_rotary", op="append", B=13, T=333, Hkv=4, D=64, page=32,
             dtype="fp16", cache="fp16", rot=64, interleaved=False, len_min=340, len_max=1500,
             ragged=True),
        # an 8-bit cache of 8 sequences read back for a dense prefill
        dict(name="gather_q8_batch", op="gather", B=8, Hkv=8, D=128, page=16, cache="e4m3",
             out="bf16", len_min=2048, len_max=8192),
        # one odd-length sequence read back in fp32
        dict(name="gather_q8_one_fp32", op="gather", B=1, Hkv=2, D=256, page=64, cache="e4m3",
             out="fp32", len_min=1021, len_max=1021),
        # decode of 128 sequences of 1K to 4K tokens over the 8-bit cache, one token each
        dict(name="decode_q8_batch", op="tree", B=128, T=1, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="e4m3", len_min=1024, len_max=4096, masked=False, ragged=False),
        # 64 drafted tokens a sequence over the 8-bit cache
        dict(name="tree_q8_64", op="tree", B=16, T=64, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
             cache="e4m3", len_min=2048, len_max=8192, masked=True, ragged=True),
        # 16 drafted tokens a sequence over a 16-bit cache
        dict(name="tree_bf16_16", op="tree", B=32, T=16, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", len_min=1024, len_max=4096, masked=True, ragged=False),
        # one user: a small odd tree at the end of one long sequence, multi-query heads
        dict(name="tree_one_long_q8", op="tree", B=1, T=7, Hq=8, Hkv=1, D=256, page=32,
             dtype="fp16", cache="e4m3", len_min=16333, len_max=16333, masked=True, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "gather", "tree", "tree"])
    D = rng.choice([64, 128, 256])
    if op == "rotary":
        Hk, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 80, 128, 192, 256])
        rot = rng.choice([D, D // 32 * 16])
        tokens = _log_int(rng, 1, max(2, 16384 * 40 * 128 // (Hk * (G + 1) * D * 2)))
        tokens = min(tokens, 40000)
        B = min(tokens, _log_int(rng, 1, 64))
        return dict(op=op, B=B, T=max(1, tokens // B), Hq=Hk * G, Hk=Hk, D=D, rot=rot,
                    interleaved=rng.random() < 0.5, transpose=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    scaling=rng.choice(["none", "linear", "by_parts"]),
                    far=_log_int(rng, 2048, 1 << 20))
    Hkv, page = rng.choice([1, 2, 4, 8]), rng.choice([8, 16, 32, 64])
    if op == "append":
        dtype = rng.choice(["bf16", "fp16"])
        cache = rng.choice(["e4m3", dtype])
        tokens = _log_int(rng, 1, min(4096, 3100000 // (Hkv * D)))
        B = min(tokens, _log_int(rng, 1, 128))
        T = max(1, tokens // B)
        lo = T + _log_int(rng, 1, 2048)
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, page=page, dtype=dtype, cache=cache,
                    rot=rng.choice([0, D, D // 2]) if cache != "e4m3" else 0,
                    interleaved=rng.random() < 0.5, len_min=lo,
                    len_max=min(lo + rng.randrange(0, 2048), max(lo, 100000 // B)),
                    ragged=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp16"])
    cache = rng.choice(["e4m3", "e4m3", dtype])
    if op == "gather":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 3, max(4, min(16384, 35000000 // (B * Hkv * D))))
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, cache=cache,
                    out=rng.choice(["bf16", "fp16", "fp32"]) if cache == "e4m3" else dtype,
                    len_min=rng.randrange(1, hi + 1), len_max=hi)
    B, T, G = _log_int(rng, 1, 128), _log_int(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
    most = min(16384, 170000000 // (B * Hkv * D), 13000000000 // (B * T * Hkv * G * D))
    hi = max(T, _log_int(rng, 1, max(2, most)))
    return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, dtype=dtype, cache=cache,
                len_min=max(T, rng.randrange(1, hi + 1)), len_max=hi, masked=rng.random() < 0.7,
                ragged=rng.random() < 0.3)


def _spread(n, lo, hi):
    """n lengths over lo..hi, the same for every seed (the work of a case is then known)."""
    return [lo + int((hi - lo) * ((i * GOLDEN + 0.5) % 1.0) + 0.5) for i in range(n)]


def _lens(case):
    return _spread(case["B"], case["len_min"], case["len_max"])


def _new_lens(case):
    """New (or drafted) tokens of each sequence: all T, or from one on where ragged."""
    B, T = case["B"], case["T"]
    return _spread(B, 1, T) if case["ragged"] else [T] * B


def _frequencies(rot, scaling, device):
    """Inverse frequencies in 64 bits and the amplitude that goes with them."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "by_parts":  # YaRN: long wavelengths interpolated, short ones kept
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return (1 - keep) * f / 32.0 + keep * f, 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _pool(gen, case, pages, dtype):
    """A cache pool in use: every slot holds some earlier token's values."""
    shape = (pages, case["Hkv"], case["page"], case["D"])
    dev = "cuda"
    if dtype == torch.float8_e4m3fn:
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
        x = (x * 110.0).clamp(-448, 448).to(dtype)
        s = torch.randint(118, 121, shape[:3], generator=gen, device=dev, dtype=torch.uint8)
        return x, s
    return torch.randn(shape, generator=gen, device=dev, dtype=dtype) * 0.5, None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    op, dev = case["op"], "cuda"
    s = {"case": case}
    if own:
        import softmax_attention_gb300  # noqa: F401  (loaded before the first call, as a program does)
    if op == "rotary":
        B, T, D, dt = case["B"], case["T"], case["D"], DTYPES[case["dtype"]]
        H = case["Hq"] + case["Hk"]
        # queries and keys as the projection leaves them: one row a token, heads side by side
        qk = torch.randn((B, T, H, D), generator=gen, device=dev, dtype=dt)
        s["q"] = qk[:, :, :case["Hq"]].transpose(1, 2)
        s["k"] = qk[:, :, case["Hq"]:].transpose(1, 2)
        start = torch.randint(0, max(1, case["far"] - T + 1), (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        s["inv_freq"], s["amplitude"] = _frequencies(case["rot"], case["scaling"], dev)
        return s
    lens = _lens(case)
    per = [-(-n // case["page"]) for n in lens]
    width = max(per) + 1
    pool = sum(per) + 3
    perm = torch.randperm(pool, generator=cpu).tolist()
    table, at = [], 0
    for n in per:
        table.append(perm[at:at + n] + [0] * (width - n))
        at += n
    s["page_table"] = torch.tensor(table, dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_len"] = max(lens)
    cache = DTYPES[case["cache"]]
    s["k_pages"], s["k_scales"] = _pool(gen, case, pool, cache)
    s["v_pages"], s["v_scales"] = _pool(gen, case, pool, cache)
    if op == "append":
        B, T, Hkv, D, dt = case["B"], case["T"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
        kv = torch.randn((B, T, 2 * Hkv, D), generator=gen, device=dev, dtype=torch.float32)
        # heads and tokens differ in size, as projections do
        kv = kv * torch.exp(torch.randn((B, T, 2 * Hkv, 1), generator=gen, device=dev))
        kv = kv.to(dt)
        s["k"] = kv[:, :, :Hkv].transpose(1, 2)
        s["v"] = kv[:, :, Hkv:].transpose(1, 2)
        s["new_lens"] = (torch.tensor(_new_lens(case), dtype=torch.int32, device=dev)
                         if case["ragged"] else None)
        if case["rot"]:
            s["inv_freq"], s["amplitude"] = _frequencies(case["rot"], "none", dev)
    if op == "tree":
        B, T, Hq, D, dt = case["B"], case["T"], case["Hq"], case["D"], DTYPES[case["dtype"]]
        s["q"] = torch.randn((B, Hq, T, D), generator=gen, device=dev, dtype=dt)
        s["draft_lens"] = (torch.tensor(_new_lens(case), dtype=torch.int32, device=dev)
                           if case["ragged"] else None)
        s["tree_mask"] = None
        if case["masked"]:
            # random trees: each token's parent is an earlier token, or the context
            words = -(-T // 64)
            mask = []
            for _ in range(B):
                rows, up = [], torch.rand(T, generator=cpu).tolist()
                for i in range(T):
                    parent = int(up[i] * (i + 1)) - 1
                    rows.append((rows[parent] if parent >= 0 else 0) | (1 << i))
                cut = [[(r >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for r in rows]
                mask.append([[x - 2 ** 64 if x >= 2 ** 63 else x for x in r] for r in cut])
            s["tree_mask"] = torch.tensor(mask, dtype=torch.int64, device=dev)
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# -------------------------------------------------------------------------------- plain forms
def _rotate(x, positions, inv_freq, amplitude, interleaved, transpose):
    """x [B,H,T,D] in fp32, its first 2 * len(inv_freq) columns rotated."""
    half = inv_freq.numel()
    angle = positions.double()[:, None, :, None] * inv_freq
    c, s = (angle.cos() * amplitude).float(), (angle.sin() * amplitude).float()
    if transpose:
        s = -s
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    ya, yb = a * c - b * s, b * c + a * s
    y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((y, rest), -1)


def _quantise(x):
    """e4m3 values and the scale bytes of x [..., D] in fp32: the least power of two that brings
    the largest value to 448 or less."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    y = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return y, (e + 127).to(torch.uint8)


def _plain_append(s):
    case = s["case"]
    B, T = case["B"], case["T"]
    dev = s["k"].device
    n = s["new_lens"] if s["new_lens"] is not None else torch.full((B,), T, device=dev)
    t = torch.arange(T, device=dev)
    pos = (s["seq_lens"] - n)[:, None] + t
    k, v = s["k"].float(), s["v"].float()
    if case["rot"]:
        k = _rotate(k, pos, s["inv_freq"], s["amplitude"], case["interleaved"], False)
    b, i = torch.nonzero(t < n[:, None], as_tuple=True)
    p = pos[b, i].long()
    page, slot = s["page_table"][b, p // case["page"]].long(), p % case["page"]
    for x, pages, scales in ((k, s["k_pages"], s["k_scales"]), (v, s["v_pages"], s["v_scales"])):
        x = x.transpose(1, 2)[b, i]
        if scales is not None:
            y, e = _quantise(x)
            pages.view(torch.uint8)[page, :, slot] = y.view(torch.uint8)
            scales[page, :, slot] = e
        else:
            pages[page, :, slot] = x.to(pages.dtype)


def _dense(s, pages, scales):
    """[B,Hkv,max_len,D] in fp32, zeros past each sequence."""
    case, L = s["case"], s["max_len"]
    ids = s["page_table"][:, :-(-L // case["page"])].long()
    if scales is not None:
        x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
        x = torch.ldexp(x, scales[ids].int()[..., None] - 127)
    else:
        x = pages[ids].float()
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :L]
    inside = torch.arange(L, device=x.device) < s["seq_lens"][:, None]
    return torch.where(inside[:, None, :, None], x, 0.0)


def _visible(s):
    """[B,T,max_len]: which keys each drafted token sees."""
    case, L, dev = s["case"], s["max_len"], s["q"].device
    B, T = case["B"], case["T"]
    n = s["draft_lens"] if s["draft_lens"] is not None else torch.full((B,), T, device=dev)
    t = torch.arange(T, device=dev)
    if s["tree_mask"] is not None:
        word, bit = t // 64, t % 64
        tree = ((s["tree_mask"][:, :, word] >> bit) & 1).bool().expand(B, T, T)
    else:
        tree = (t[None, :] <= t[:, None]).expand(B, T, T)
    key = torch.arange(L, device=dev)
    rel = key - (s["seq_lens"] - n)[:, None]
    draft = tree.gather(2, rel.clamp(0, T - 1)[:, None, :].expand(B, T, L))
    seen = torch.where(rel[:, None, :] < 0, True, draft) & (key < s["seq_lens"][:, None])[:, None, :]
    return seen & (t < n[:, None])[:, :, None]


def _plain_tree(s):
    case = s["case"]
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    k, v = _dense(s, s["k_pages"], s["k_scales"]), _dense(s, s["v_pages"], s["v_scales"])
    q = s["q"].float().view(B, Hkv, -1, T, D).flatten(2, 3) * s["scale"]
    x = (q @ k.transpose(2, 3)).view(B, Hkv, Hq // Hkv, T, -1)
    x = x.masked_fill(~_visible(s)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    out = p.flatten(2, 3) @ v
    total = total.flatten(2, 3)
    out = torch.where(total > 0, out / total, 0.0)
    lse = total.log() + m.flatten(2, 3)
    return out.view(B, Hq, T, D).to(s["q"].dtype), lse.view(B, Hq, T)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import softmax_attention_gb300 as fa
        if op == "rotary":
            return fa.fa_rotary(s["q"], s["k"], s["positions"], s["inv_freq"],
                                amplitude=s["amplitude"], interleaved=case["interleaved"],
                                transpose=case["transpose"])
        if op == "append":
            rot = {}
            if case["rot"]:
                rot = dict(inv_freq=s["inv_freq"], amplitude=s["amplitude"],
                           interleaved=case["interleaved"])
            fa.fa_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"],
                               s["seq_lens"], new_lens=s["new_lens"], k_scales=s["k_scales"],
                               v_scales=s["v_scales"], **rot)
        elif op == "gather":
            return fa.fa_cache_gather(s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"],
                                      s["max_len"], dtype=DTYPES[case["out"]],
                                      k_scales=s["k_scales"], v_scales=s["v_scales"])
        else:
            return fa.fa_tree_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                           s["seq_lens"], s["max_len"], tree_mask=s["tree_mask"],
                                           draft_lens=s["draft_lens"], scale=s["scale"],
                                           k_scales=s["k_scales"], v_scales=s["v_scales"])
    else:
        if op == "rotary":
            args = (s["positions"], s["inv_freq"], s["amplitude"], case["interleaved"],
                    case["transpose"])
            dt = s["q"].dtype
            return _rotate(s["q"], *args).to(dt), _rotate(s["k"], *args).to(dt)
        if op == "append":
            _plain_append(s)
        elif op == "gather":
            dt = DTYPES[case["out"]]
            return (_dense(s, s["k_pages"], s["k_scales"]).to(dt),
                    _dense(s, s["v_pages"], s["v_scales"]).to(dt))
        else:
            return _plain_tree(s)
    # a cache write: the pools (8-bit values and their scales) are the outputs
    out = [s["k_pages"], s["v_pages"]]
    return out + [s["k_scales"], s["v_scales"]] if s["k_scales"] is not None else out


# ---------------------------------------------------------------------------------- 64 bits
def _exact_rotary(x, positions, inv_freq, amplitude, interleaved, transpose):
    """Complex numbers turned by their angles."""
    half = inv_freq.numel()
    th = torch.einsum("bt,f->btf", positions.double(), inv_freq)
    turn = torch.polar(torch.full_like(th, amplitude), -th if transpose else th)[:, None]
    y = x.double().clone()
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(s, b, pages, scales, n):
    """The first n tokens of sequence b: [n,Hkv,D] in 64 bits."""
    t = torch.arange(n, device=pages.device)
    ps = pages.shape[2]
    page, slot = s["page_table"][b, t // ps].long(), t % ps
    if scales is None:
        return pages[page, :, slot].double()
    value = pages.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).double()
    return value * torch.pow(2.0, scales[page, :, slot].double() - 127.0)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        args = (s["positions"], s["inv_freq"], s["amplitude"], case["interleaved"],
                case["transpose"])
        return _exact_rotary(s["q"], *args), _exact_rotary(s["k"], *args)
    if op == "append":
        if case["cache"] == "e4m3":
            return None  # what an 8-bit value is rounded to is a choice, compared bit for bit
        pools = [s["k_pages"].double(), s["v_pages"].double()]
        for b, (length, n) in enumerate(zip(_lens(case), _new_lens(case))):
            k, v = s["k"][b:b + 1, :, :n].double(), s["v"][b:b + 1, :, :n].double()
            pos = torch.arange(length - n, length, device=k.device)
            if case["rot"]:
                k = _exact_rotary(k, pos[None], s["inv_freq"], s["amplitude"],
                                  case["interleaved"], False)
            page = s["page_table"][b, pos // case["page"]].long()
            for pool, x in zip(pools, (k, v)):
                pool[page, :, pos % case["page"]] = x[0].transpose(0, 1)
        return pools
    lens = _lens(case)
    if op == "gather":
        outs = []
        for pages, scales in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])):
            y = torch.zeros((case["B"], case["Hkv"], s["max_len"], case["D"]), device="cuda",
                            dtype=torch.float64)
            for b, n in enumerate(lens):
                y[b, :, :n] = _exact_rows(s, b, pages, scales, n).transpose(0, 1)
            outs.append(y)
        return tuple(outs)
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, (length, n) in enumerate(zip(lens, _new_lens(case))):
        k = _exact_rows(s, b, s["k_pages"], s["k_scales"], length)
        v = _exact_rows(s, b, s["v_pages"], s["v_scales"], length)
        q = s["q"][b, :, :n].double().reshape(Hkv, Hq // Hkv, n, D)
        x = torch.einsum("hgtd,jhd->hgtj", q, k) * s["scale"]
        j = torch.arange(n, device="cuda")
        if s["tree_mask"] is None:
            hidden = j[None, :] > j[:, None]
        else:
            words = s["tree_mask"][b].cpu().tolist()
            hidden = torch.tensor([[not (words[i][c // 64] >> (c % 64)) & 1 for c in range(n)]
                                   for i in range(n)], device="cuda")
        x[..., length - n:] = x[..., length - n:].masked_fill(hidden, -math.inf)
        lse[b, :, :n] = torch.logsumexp(x, -1).reshape(Hq, n)
        w = torch.softmax(x, -1)
        out[b, :, :n] = torch.einsum("hgtj,jhd->hgtd", w, v).reshape(Hq, n, D)
    return out, lse


def work(case):
    op = case["op"]
    if op == "rotary":
        tokens = case["B"] * case["T"]
        rows = tokens * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * rows * case["D"] * SIZE[case["dtype"]] + 4 * tokens + 4 * case["rot"],
                "flops": 3 * rows * case["rot"]}
    size = SIZE[case["cache"]]
    row = case["Hkv"] * (case["D"] * size + (1 if case["cache"] == "e4m3" else 0))
    if op == "append":
        tokens = sum(_new_lens(case))
        return {"bytes": 2 * tokens * (case["Hkv"] * case["D"] * SIZE[case["dtype"]] + row),
                "flops": 4 * tokens * case["Hkv"] * case["D"]}
    lens = _lens(case)
    pages = sum(-(-n // case["page"]) for n in lens)
    if op == "gather":
        dense = case["B"] * max(lens) * case["Hkv"] * case["D"] * SIZE[case["out"]]
        return {"bytes": 2 * (sum(lens) * row + dense) + 4 * pages,
                "flops": 2 * sum(lens) * case["Hkv"] * case["D"]}
    queries = case["B"] * case["Hq"] * case["T"]
    pairs = sum(n * m for n, m in zip(lens, _new_lens(case))) * case["Hq"]
    return {"bytes": 2 * sum(lens) * row + 4 * pages
            + queries * (2 * case["D"] * SIZE[case["dtype"]] + 4),
            "flops": 4 * pairs * case["D"]}
