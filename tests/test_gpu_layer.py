"""The packed-prompt operators together, as a model's attention layer uses them: norms with rotary
positions, attention and the gradients of both; and a prompt followed by a decode step."""
import math

import pytest
import torch

import softmax_attention_gb300 as fa

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    yield
    assert fa.fa_get_device_status() == fa.FA_OK, fa.fa_last_error()


def _turn(x, pos, f):
    """x [T,H,D] in 64 bits, all columns turned, half layout."""
    half = x.shape[-1] // 2
    th = pos.double()[:, None, None] * f
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * th.cos() - b * th.sin(), b * th.cos() + a * th.sin()), -1)


def _layer(q, k, v, wq, wk, pos, f, cu, scale):
    """In 64 bits, differentiable."""
    norm = lambda x, w: x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w  # noqa: E731
    q, k = _turn(norm(q, wq), pos, f), _turn(norm(k, wk), pos, f)
    G = q.shape[1] // k.shape[1]
    outs = []
    for a, b in zip(cu, cu[1:]):
        x = torch.einsum("igd,jgd->gij", q[a:b], k[a:b].repeat_interleave(G, 1)) * scale
        x = x.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), -math.inf)
        outs.append(torch.einsum("gij,jgd->igd", torch.softmax(x, -1), v[a:b].repeat_interleave(G, 1)))
    return torch.cat(outs)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2)])
def test_training_step_of_a_layer(D, Hq, Hkv):
    g = torch.Generator().manual_seed(D)
    lens = [70, 1, 133, 40]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1]
    x = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * 2).to(BF)
    w = (1 + 0.2 * torch.randn(2, D, generator=g)).to(BF)
    do = torch.randn(T, Hq, D, generator=g).to(BF)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
    f, _ = fa.rotary_frequencies(D)
    scale = 1.0 / math.sqrt(D)

    dev = x.cuda()
    qkv = [dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]]
    view = lambda t: t.transpose(0, 1)[None]  # noqa: E731  [T,H,D] as [1,H,T,D]
    wd, posd, fd, cud = w.cuda(), pos.cuda()[None], f.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda")
    q = torch.empty(T, Hq, D, dtype=BF, device="cuda")
    k = torch.empty(T, Hkv, D, dtype=BF, device="cuda")
    fa.fa_qk_norm_rotary(view(qkv[0]), view(qkv[1]), posd, fd, wd[0], wd[1], eps=EPS, q_out=view(q), k_out=view(k))
    out, lse = fa.fa_prefill_packed(q, k, qkv[2], cud, scale=scale)
    dqkv = torch.empty_like(dev)  # the projection's gradient, written in place of its slices
    dq, dk, dv = dqkv[:, :Hq], dqkv[:, Hq:Hq + Hkv], dqkv[:, Hq + Hkv:]
    fa.fa_prefill_packed_backward(do.cuda(), q, k, qkv[2], out, lse, cud, scale=scale, dq=dq, dk=dk, dv=dv)
    _, _, dwq, dwk = fa.fa_qk_norm_rotary_backward(view(dq), view(dk), view(qkv[0]), view(qkv[1]), posd, fd, wd[0],
                                                   wd[1], eps=EPS, dq=view(dq), dk=view(dk))
    torch.cuda.synchronize()

    leaves = [t.double().requires_grad_() for t in (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w[0], w[1])]
    want = _layer(*leaves, pos, f, cu, scale)
    grads = torch.autograd.grad(want, leaves, do.double())
    # In the 2-norm, relative.  Roundings to bf16 (2^-8 at most, 2^-8 / sqrt(3) in the mean square) that a result
    # goes through: q and k after the norm, which move a score s by 2^-8 sqrt(2 / 3) |s|-like amounts; P;
    # out; dS; dq and dk on their way to the norm's gradient; the result itself.  Eight of them, taken as if
    # they all pulled one way: 8 * 2^-8 / sqrt(3) = 1.8 %.
    for name, a, b in zip(("out", "dq", "dk", "dv", "dwq", "dwk"), (out, dq, dk, dv, dwq, dwk), (want, *grads)):
        off = (a.double().cpu() - b.detach()).norm() / b.detach().norm()
        assert off <= 8 * 2.0 ** -8 / math.sqrt(3), (name, off.item())


@pytest.mark.parametrize("quantised", [False, True])
def test_a_prompt_and_its_next_token(quantised):
    """Prompts of different lengths through the packed call, their keys into the paged cache, then a token
    of each by the decode call: what the packed call gives for that token at the end of the prompt."""
    g = torch.Generator().manual_seed(3)
    lens, Hq, Hkv, D, ps = [33, 1, 150], 8, 2, 128, 16
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, B = cu[-1], len(lens)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(BF).cuda()
    w = torch.ones(2, D, dtype=BF, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    f, _ = fa.rotary_frequencies(D, device="cuda")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    view = lambda t: t.transpose(0, 1)[None]  # noqa: E731
    q, k = (torch.empty(T, h, D, dtype=BF, device="cuda") for h in (Hq, Hkv))
    fa.fa_qk_norm_rotary(view(x[:, :Hq]), view(x[:, Hq:Hq + Hkv]), pos[None], f, w[0], w[1], q_out=view(q), k_out=view(k))
    v = x[:, Hq + Hkv:]
    out, lse = fa.fa_prefill_packed(q, k, v, cud)
    # the cache, prompt by prompt, all tokens but the last; then one step for the last tokens
    pages = [-(-n // ps) for n in lens]
    table = torch.zeros(B, max(pages), dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    table = table.cuda()
    dt = torch.float8_e4m3fn if quantised else BF
    kp = torch.zeros(at, Hkv, ps, D, dtype=dt, device="cuda")
    vp = torch.zeros_like(kp)
    scales = {}
    if quantised:
        scales = dict(k_scales=torch.zeros(at, Hkv, ps, dtype=torch.uint8, device="cuda"),
                      v_scales=torch.zeros(at, Hkv, ps, dtype=torch.uint8, device="cuda"))
    for b, n in enumerate(lens):
        if n > 1:
            rows = slice(cu[b], cu[b + 1] - 1)
            fa.fa_cache_append(view(k[rows]), view(v[rows]), kp, vp, table[b:b + 1].contiguous(),
                               torch.tensor([n - 1], dtype=torch.int32, device="cuda"), **scales)
    last = torch.tensor([n - 1 for n in cu[1:]], device="cuda")
    step = lambda t: t[last][:, :, None]  # noqa: E731  [B,H,1,D]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fa.fa_cache_append(step(k), step(v), kp, vp, table, seq, **scales)
    o, l = fa.fa_tree_decode_paged(step(q), kp, vp, table, seq, max(lens), **scales)
    if quantised:
        # keys and values off by up to 2^-4 of themselves, at random over 128 columns and the keys
        assert (o[:, :, 0].float() - out[last].float()).abs().max() < 0.25
        assert (l[:, :, 0] - lse[last]).abs().max() < 0.25
    else:
        torch.testing.assert_close(o[:, :, 0].float(), out[last].float(), rtol=2 * 2.0 ** -8, atol=2 * 2.0 ** -8)
        torch.testing.assert_close(l[:, :, 0], lse[last], rtol=1e-6, atol=2e-5)
