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
    [n,n] (query, drafted token) or None for a chain.  Returns, in fp64, out, lse, and what the
    error bounds need: sum_j w_j |v_j| (as out), the largest scale sum_d |q_d k_d| of a row (as lse) and sum_j |v_j|.  Hidden keys take no part at all, whatever they hold."""
    B, Hq, T, D = q.shape
    out = torch.zeros(B, Hq, T, D, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    mean_abs, sum_abs = torch.zeros_like(out), torch.zeros_like(out)
    reach = torch.zeros(B, Hq, T, dtype=torch.float64)
    for b in range(B):
        n, L = draft_lens[b], k_rows[b].shape[0]
        G = Hq // k_rows[b].shape[1]
        for i in range(n):
            seen = torch.ones(L, dtype=torch.bool)
            seen[L - n:] = torch.arange(n) <= i if mask is None else mask[b][i, :n]
            if not seen.any():
                continue
            k, v = k_rows[b][seen], v_rows[b][seen]
            for h in range(Hq):
                x = q[b, h, i].double().cpu()
                s = (k[:, h // G] @ x) * scale
                m = s.max()
                if m == -math.inf:
                    continue
                w = (s - m).exp()
                out[b, h, i] = (w[:, None] * v[:, h // G]).sum(0) / w.sum()
                lse[b, h, i] = m + w.sum().log()
                mean_abs[b, h, i] = (w[:, None] * v[:, h // G].abs()).sum(0) / w.sum()
                sum_abs[b, h, i] = v[:, h // G].abs().sum(0)
                reach[b, h, i] = (k[:, h // G].abs() @ x.abs()).max() * abs(scale)
    return out, lse, mean_abs, reach, sum_abs


def check_tree(out, lse, want, dtype, D, what=""):
    """The kernel's out and lse against tree_attention's.

    A score is a sum of D products of 16-bit values in fp32, in the tensor core's own order and
    with its own truncation: each of the D additions is off by at most 2^-23 of the running
    sum, which sum |q_d k_d| bounds; times the scale, minus the maximum, through 2^x (2^-22):
    delta below bounds the relative error of a weight, once in the numerator and once in the
    sum.  A weight is rounded to dtype on its way into the second product (half a step), the
    output once at its end.  An fp16 weight below 2^-14 has an absolute rounding, 2^-25, of a
    weight held 2^7 times larger, where the row's largest is at least 1 (and so the sum by
    which it is divided): 2^-32 sum_j |v_j| in all."""
    o, l, mean_abs, reach, sum_abs = want
    out, lse = out.double().cpu(), lse.double().cpu()
    half = torch.finfo(dtype).eps / 2
    delta = (D + 8) * 2.0 ** -23 * reach + 2.0 ** -20
    tiny = torch.finfo(dtype).tiny
    bound = (half + 2 * delta[..., None]) * mean_abs + half * o.abs() + tiny
    if dtype == torch.float16:
        bound = bound + 2.0 ** -32 * sum_abs
    empty = l == -math.inf
    assert torch.equal(empty, lse == -math.inf), f"{what}: other rows are empty"
    assert (out[empty] == 0).all(), f"{what}: empty rows"
    fin = torch.isfinite(o)
    assert torch.equal(torch.isnan(o), torch.isnan(out)), f"{what}: NaN elsewhere"
    bad = ((out - o).abs() > bound) & fin
    assert not bad.any(), f"{what}: {int(bad.sum())} off, {((out - o).abs() / bound)[fin].max():.2f} of the bound"
    dl = (lse - l).abs()[~empty & torch.isfinite(l)]
    bl = (delta + 2.0 ** -21 * l.abs())[~empty & torch.isfinite(l)]
    assert (dl <= bl).all(), f"{what}: lse off by {(dl / bl).max():.2f} of the bound"
