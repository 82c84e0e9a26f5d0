"""Plain 64-bit forms of block selection, block-sparse attention and 8-bit checkpoints, and the
error bounds that follow from the roundings the kernels make (torch, on the inputs' device).

Roundings counted: half a step of bf16 is 2^-8 relative.  P and dS enter their products in
bf16, results are rounded once to bf16; everything else is fp32.  SLACK covers the fp32 part
relative to a row's terms: a score is a sum of D <= 128 products accumulated in fp32, off by at
most D 2^-24 scale sum|q||k|, and scale sum|q||k| stays below 16 for the unit normals used here
(mean 0.64 sqrt(D), largest seen about 1.5 times that), so the exponent is off by at most
128 * 2^-24 * 16 = 1.3e-4, which with the exponential's and the row sum's own errors (2^-21)
stays under 3e-4."""
import math

import torch

HALF = 2.0 ** -8   # half a step of bf16, relative
SLACK = 3e-4


def limits(B, Sq, Sk, causal, kv_len=None, q_start=None, device="cpu"):
    """Keys that query i of batch entry b may see, [B,Sq]."""
    n = torch.full((B,), Sk, device=device) if kv_len is None else kv_len.to(device).long().clamp(0, Sk)
    s = torch.full((B,), Sk - Sq, device=device) if q_start is None else q_start.to(device).long()
    lim = n[:, None].expand(B, Sq)
    if causal:
        lim = torch.minimum(lim, (s[:, None] + torch.arange(Sq, device=device) + 1).clamp(min=0))
    return lim


def means(k, block, kv_len=None):
    B, Hkv, Sk, D = k.shape
    nb = -(-Sk // block)
    out = torch.zeros(B, Hkv, nb, D, dtype=torch.float64, device=k.device)
    for b in range(B):
        n = Sk if kv_len is None else min(max(int(kv_len[b]), 0), Sk)
        for j in range(-(-n // block)):
            out[b, :, j] = k[b, :, j * block:min((j + 1) * block, n)].double().mean(1)
    return out


def select(q, mean, Sk, block, topk, causal, sink, local, kv_len=None, q_start=None):
    """By the definition, one query at a time."""
    B, H, Sq, D = q.shape
    Hkv, nb = mean.shape[1:3]
    out = torch.full((B, Hkv, Sq, topk), -1, dtype=torch.int32)
    lim = limits(B, Sq, Sk, causal, kv_len, q_start, "cpu")
    qs = q.double().unflatten(1, (Hkv, H // Hkv)).sum(2)
    score = torch.einsum("bhid,bhjd->bhij", qs, mean.double()).cpu()
    for b in range(B):
        for h in range(Hkv):
            for i in range(Sq):
                n = -(-int(lim[b, i]) // block)
                forced = {j for j in range(n) if j < sink or j >= n - local}
                rest = sorted((j for j in range(n) if j not in forced),
                              key=lambda j: (-float(score[b, h, i, j]), j))
                pick = sorted(list(forced)[:topk] + rest[:max(0, topk - len(forced))])
                out[b, h, i, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return out


def mask(idx, Sk, block, lim):
    """[B,Hkv,Sq,Sk]: the keys each query attends to."""
    nb = -(-Sk // block)
    ok = (idx >= 0) & (idx < nb)
    on = torch.zeros(*idx.shape[:3], nb + 1, dtype=torch.bool, device=idx.device)
    on.scatter_(3, torch.where(ok, idx, nb).long(), True)
    on = on[..., :nb].repeat_interleave(block, dim=3)[..., :Sk]
    return on & (torch.arange(Sk, device=idx.device) < lim.to(idx.device)[:, None, :, None])


def forward(q, k, v, m, scale=None):
    """(o, lse, bound on o) under the mask m [B,Hkv,Sq,Sk]."""
    B, H, Sq, D = q.shape
    Hkv = k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    any_key = m.any(2)  # a key that nobody attends to is left out, whatever it holds
    kd = torch.where(any_key[..., None], k.double(), 0.0)
    vd = torch.where(any_key[..., None], v.double(), 0.0)
    qd = q.double().unflatten(1, (Hkv, H // Hkv))
    x = torch.einsum("bhgid,bhjd->bhgij", qd, kd) * scale
    x = x.masked_fill(~m[:, :, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.where(lse[..., None] == -math.inf, 0.0, torch.exp(x - lse[..., None]))
    o = torch.einsum("bhgij,bhjd->bhgid", p, vd).flatten(1, 2)
    a = torch.einsum("bhgij,bhjd->bhgid", p, vd.abs()).flatten(1, 2)
    return o, lse.flatten(1, 2), (HALF + SLACK) * a + HALF * o.abs()


def backward(q, k, v, o, do, lse, m, scale=None):
    """((dq, dk, dv), their bounds) from the forward's rounded o and lse."""
    B, H, Sq, D = q.shape
    Hkv = k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    any_key = m.any(2)
    kd = torch.where(any_key[..., None], k.double(), 0.0)
    vd = torch.where(any_key[..., None], v.double(), 0.0)
    g = lambda t: t.double().unflatten(1, (Hkv, H // Hkv))
    qd, od, dod = g(q), g(o), g(do)
    x = torch.einsum("bhgid,bhjd->bhgij", qd, kd) * scale
    p = torch.where(m[:, :, None], torch.exp(x - g(lse)[..., None]), 0.0)
    dp = torch.einsum("bhgid,bhjd->bhgij", dod, vd)
    ds = p * (dp - (dod * od).sum(-1, keepdim=True))
    # fp32 sums of D products: dP and delta
    eps = D * 2.0 ** -24 * (torch.einsum("bhgid,bhjd->bhgij", dod.abs(), vd.abs())
                            + (dod * od).abs().sum(-1, keepdim=True))
    dsb = (HALF + SLACK) * ds.abs() + p * eps
    dq = scale * torch.einsum("bhgij,bhjd->bhgid", ds, kd)
    dk = scale * torch.einsum("bhgij,bhgid->bhjd", ds, qd)
    dv = torch.einsum("bhgij,bhgid->bhjd", p, dod)
    bq = scale * torch.einsum("bhgij,bhjd->bhgid", dsb, kd.abs()) + HALF * dq.abs()
    bk = scale * torch.einsum("bhgij,bhgid->bhjd", dsb, qd.abs()) + HALF * dk.abs()
    bv = (HALF + SLACK) * torch.einsum("bhgij,bhgid->bhjd", p, dod.abs()) + HALF * dv.abs()
    return (dq.flatten(1, 2), dk, dv), (bq.flatten(1, 2), bk, bv)


def within(got, want, bound, tiny=1e-6):
    """The largest |got - want| over its bound; `tiny` absorbs sums that cancel to nothing."""
    d = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all()
    return float((d / (bound + tiny)).max()) if d.numel() else 0.0


def ckpt_pack(x):
    """(m, e) of the 8-bit form in 64 bits."""
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    bad = ~torch.isfinite(top)
    # frexp: top = f 2^n with f in [1/2, 1), so floor(log2 top) = n - 1
    e = torch.where(top > 0, torch.frexp(torch.where(bad, 1.0, top)).exponent - 7, -126).clamp(min=-126)
    step = ((e.long() + 1023) << 52).view(torch.float64)
    m = (torch.where(bad[..., None], 0.0, g) / step[..., None]).round().clamp(-127, 127)
    e = torch.where(bad, -128, e)
    return m.flatten(-2).to(torch.int8), e.to(torch.int8)


def ckpt_values(m, e):
    step = ((e.long().clamp(min=-126) + 1023) << 52).view(torch.float64)
    step = torch.where(e == -128, math.nan, step)
    return (m.double().unflatten(-1, (-1, 32)) * step[..., None]).flatten(-2)
