"""Plain 64-bit references of rotary positions and the paged cache, for the tests.

Written from the definitions in include/fa.h, on the CPU, one row after another where that is
the plainest; nothing of the library is used.
"""
import math

import torch


def rotate(x, positions, inv_freq, amplitude=1.0, interleaved=False, transpose=False):
    """x [B,H,T,D] (any dtype) -> fp64."""
    x = x.double().cpu()
    f = inv_freq.double().cpu()
    half = f.numel()
    th = positions.cpu().double()[:, None, :, None] * f * (-1.0 if transpose else 1.0)
    a_cols = torch.arange(half) * 2 if interleaved else torch.arange(half)
    b_cols = a_cols + (1 if interleaved else half)
    y = x.clone()
    a, b = x[..., a_cols], x[..., b_cols]
    y[..., a_cols] = amplitude * (a * th.cos() - b * th.sin())
    y[..., b_cols] = amplitude * (b * th.cos() + a * th.sin())
    return y


def pair_sum(x, inv_freq, interleaved=False):
    """|x_a| + |x_b| of each element's pair (0 outside the rotated part), fp64."""
    half = inv_freq.numel()
    x = x.double().cpu().abs()
    s = torch.zeros_like(x)
    a = torch.arange(half) * 2 if interleaved else torch.arange(half)
    b = a + (1 if interleaved else half)
    s[..., a] = s[..., b] = x[..., a] + x[..., b]
    return s


def exponent(amax: float) -> int:
    """The least e >= -126 with amax <= 448 * 2^e."""
    e = -126
    if amax > 0:
        e = max(-126, math.frexp(amax / 448.0)[1] - 2)
        while amax > math.ldexp(448.0, e):
            e += 1
    return e


# every non-negative finite e4m3 value, in order
_E4M3 = torch.tensor([m / 512.0 for m in range(8)] +
                     [(1 + m / 8.0) * 2.0 ** (k - 7) for k in range(1, 16) for m in range(8)][:-1],
                     dtype=torch.float64)


def quantise(x):
    """x [..., D] -> (codes uint8, bytes uint8): the 8-bit row format, to nearest even."""
    x = x.double().cpu()
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    amax = fin.amax(-1)
    e = torch.tensor([exponent(v) for v in amax.flatten().tolist()],
                     dtype=torch.int64).view(amax.shape)
    mag = (x.abs() * torch.pow(2.0, -e.double())[..., None]).clamp(max=448.0)
    mag = torch.nan_to_num(mag, nan=0.0)
    hi = torch.searchsorted(_E4M3, mag.contiguous()).clamp(max=_E4M3.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = _E4M3[hi] - mag, mag - _E4M3[lo]
    code = torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))
    code = torch.where(torch.isnan(x), torch.full_like(code, 0x7F), code)
    sign = torch.signbit(x)
    code = code + 128 * sign
    return code.to(torch.uint8), (e + 127).to(torch.uint8)


def dequantise(codes, scales):
    """fp64 values of uint8 codes [..., D] and scale bytes [...]."""
    table = torch.cat((_E4M3, torch.tensor([math.nan], dtype=torch.float64)))
    table = torch.cat((table, -table))
    v = table[codes.cpu().long()]
    return v * torch.pow(2.0, scales.cpu().double() - 127.0)[..., None]


def make_table(lens, page_size, num_pages, gen, spare=2):
    """A page table of distinct random pages; entries past a sequence are -1."""
    per = [-(-n // page_size) for n in lens]
    perm = torch.randperm(num_pages, generator=gen).tolist()
    assert sum(per) <= num_pages
    table = torch.full((len(lens), max(per + [0]) + spare), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    return table


def rows_of(pages, table, b, n):
    """Tokens 0..n-1 of sequence b: [n, Hkv, ...] of pages [P, Hkv, page_size, ...]."""
    ps = pages.shape[2]
    t = torch.arange(n)
    return pages[table[b, t // ps].long(), :, t % ps]


def tree_attention(q, k_rows, v_rows, draft_lens, mask, scale):
    """q [B,Hq,T,D]; k_rows, v_rows: per sequence [len,Hkv,D] fp64; mask: per sequence a boolean
    [n,n] (query, drafted token) or None for a chain.  Returns out, lse in fp64; hidden keys
    take no part at all, whatever they hold."""
    B, Hq, T, D = q.shape
    out = torch.zeros(B, Hq, T, D, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    for b in range(B):
        n, L = draft_lens[b], k_rows[b].shape[0]
        G = Hq // k_rows[b].shape[1] if L else 1
        for i in range(n):
            seen = torch.ones(L, dtype=torch.bool)
            tail = torch.arange(n) <= i if mask is None else mask[b][i, :n]
            seen[L - n:] = tail
            if not seen.any():
                continue
            k, v = k_rows[b][seen], v_rows[b][seen]
            for h in range(Hq):
                s = (k[:, h // G] @ q[b, h, i].double().cpu()) * scale
                m = s.max()
                if m == -math.inf:
                    continue
                w = (s - m).exp()
                out[b, h, i] = (w[:, None] * v[:, h // G]).sum(0) / w.sum()
                lse[b, h, i] = m + w.sum().log()
    return out, lse
