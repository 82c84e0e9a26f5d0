"""Measured cases of block selection, block-sparse attention and 8-bit checkpoints.

``run`` computes each operator in elementary torch operations, or, where ``own`` is
set, through the package's entry points.  Shapes follow the package's layouts:
q, o [B,H,Sq,D], k, v [B,Hkv,Sk,D], lse [B,H,Sq], selected blocks [B,Hkv,Sq,topk].
"""
import math

import torch

own = False

GROUP = 32  # elements that share an exponent in an 8-bit checkpoint


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a training prompt's selection: every query of a 16k sequence, grouped heads
        dict(name="select_prompt_16k", op="select", B=1, H=16, Hkv=4, Sq=16384, Sk=16384, D=128, block=64,
             topk=16, ragged=False),
        # a chunk of a prompt behind a cached prefix, sequences of unlike length, blocks of 128
        dict(name="select_chunk_ragged", op="select", B=2, H=8, Hkv=8, Sq=1999, Sk=5003, D=64, block=128,
             topk=9, ragged=True),
        # one new token of 64 sequences: its block's mean is brought up to date, then blocks are picked
        dict(name="select_tokens_b64", op="select", B=64, H=32, Hkv=8, Sq=1, Sk=16384, D=128, block=64,
             topk=16, ragged=True),
        # a training step (forward and backward) of an 8k layer with four query heads per K/V head
        dict(name="sparse_train_gqa_8k", op="train", B=1, H=16, Hkv=4, Sq=8192, Sk=8192, D=128, block=64,
             topk=16, ragged=False),
        # a training step of a 16k layer whose heads select for themselves, D = 64, larger blocks
        dict(name="sparse_train_mha_16k", op="train", B=1, H=8, Hkv=8, Sq=16384, Sk=16384, D=64, block=128,
             topk=8, ragged=False),
        # a prompt's chunk over a cached prefix, odd lengths, forward only
        dict(name="sparse_prompt_ragged", op="attend", B=2, H=16, Hkv=2, Sq=1501, Sk=6007, D=128, block=64,
             topk=16, ragged=True),
        # the smallest call: one token of one sequence, where latency counts
        dict(name="sparse_token_b1", op="attend", B=1, H=32, Hkv=8, Sq=1, Sk=4096, D=128, block=64,
             topk=16, ragged=False),
        # one token of each of 64 sequences
        dict(name="sparse_tokens_b64", op="attend", B=64, H=32, Hkv=8, Sq=1, Sk=16384, D=128, block=64,
             topk=16, ragged=True),
        # checkpoints of a small layer's q, k, v, o: written and read back
        dict(name="ckpt_small", op="ckpt", B=1, H=8, Hkv=2, Sq=300, Sk=300, D=64),
        # checkpoints of a causal 8k layer's q, k, v, o
        dict(name="ckpt_8k", op="ckpt", B=2, H=32, Hkv=32, Sq=8192, Sk=8192, D=128),
        # the dense backward of a full-mask 4k layer from its checkpoints
        dict(name="ckpt_bwd_full_4k", op="ckpt_bwd", B=2, H=16, Hkv=16, Sq=4096, Sk=4096, D=128, causal=False),
        # the dense backward of a causal 8k layer with grouped heads from its checkpoints
        dict(name="ckpt_bwd_causal_gqa_8k", op="ckpt_bwd", B=1, H=16, Hkv=4, Sq=8192, Sk=8192, D=64, causal=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select_token", "train", "attend", "token", "ckpt", "ckpt_bwd"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    block = rng.choice([64, 128, 256])
    topk = rng.randint(3, 1024 // block + 4)
    c = dict(B=1, H=Hkv * G, Hkv=Hkv, D=D, block=block, topk=topk)
    if op in ("select", "attend"):
        c["Sk"] = _log_int(rng, 200, 8192)
        c["Sq"] = min(c["Sk"], _log_int(rng, 2, 4096))
        c["B"] = rng.choice([1, 2, 3])
        c["H"] = min(c["H"], 16 // Hkv * Hkv)
        return dict(c, op=op, ragged=rng.random() < 0.5)
    if op in ("select_token", "token"):
        c["Sk"] = _log_int(rng, 100, 16384)
        c["B"] = _log_int(rng, 1, 64)
        return dict(c, op="select" if op == "select_token" else "attend", Sq=1, ragged=rng.random() < 0.7)
    if op == "train":
        Hkv = c["Hkv"] = min(Hkv, 4)
        c["H"] = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * Hkv <= 8])
        c["Sq"] = c["Sk"] = _log_int(rng, 100, 8192)
        return dict(c, op="train", ragged=False)
    if op == "ckpt":
        c["Sq"] = c["Sk"] = _log_int(rng, 1, 8192)
        c["B"] = rng.choice([1, 2])
        return dict(B=c["B"], H=min(c["H"], 32), Hkv=Hkv, D=D, Sq=c["Sq"], Sk=c["Sk"], op="ckpt")
    H = rng.choice([4, 8, 16])
    S = 256 * rng.randint(1, 24)
    causal = rng.random() < 0.5
    return dict(op="ckpt_bwd", B=1, H=H, Hkv=rng.choice([H, H // 2, H // 4]), Sq=S, Sk=S, D=D, causal=causal)


# ------------------------------------------------------------------ inputs
def _positions(case, gen):
    """Lengths of the sequences and positions of their first query (None: all full)."""
    B, Sq, Sk = case["B"], case["Sq"], case["Sk"]
    if not case["ragged"]:
        return None, None
    n = torch.randint(max(Sq, Sk // 2), Sk + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    return n, n - Sq


def _limits(s):
    """Keys that query i of batch b may see, [B,Sq] (causal)."""
    B, Sq, Sk = s["B"], s["Sq"], s["Sk"]
    i = torch.arange(Sq, device="cuda")
    if s["kv_len"] is None:
        return (i + (Sk - Sq) + 1).expand(B, Sq)
    return torch.minimum(s["q_start"][:, None] + i + 1, s["kv_len"][:, None]).clamp(min=0).long()


def _pick(score, limit, block, topk):
    """Block numbers [..,Sq,topk] by the selection's rule: the first and the last visible
    block, then the best scores, ties to the lower block; ascending, then -1."""
    nb = score.shape[-1]
    j = torch.arange(nb, device=score.device)
    nvis = (limit + block - 1) // block
    nvis = nvis[:, None, :, None]
    visible = j < nvis
    forced = visible & ((j < 1) | (j >= nvis - 1))
    s = torch.where(forced, math.inf, score).masked_fill(~visible, -math.inf)
    order = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :topk]
    if topk > nb:
        order = torch.nn.functional.pad(order, (0, topk - nb), value=nb)
    order = torch.where(order < nvis, order, nb).sort(dim=-1).values
    return torch.where(order < nb, order, -1).to(torch.int32)


def _power(e):
    """2^e in fp32 for -126 <= e <= 127, without a rounding (halves are common below)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _pack(x):
    """Checkpoint of x in the stored form: int8 mantissas and exponents of groups of 32."""
    g = x.float().unflatten(-1, (-1, GROUP))
    e = (torch.frexp(g.abs().amax(-1)).exponent - 7).clamp(min=-126)
    m = (g * _power(-e)[..., None]).round().clamp(-127, 127)
    return m.flatten(-2).to(torch.int8), e.to(torch.int8)


def _values(m, e):
    """The fp32 values that a checkpoint stands for."""
    return (m.float().unflatten(-1, (-1, GROUP)) * _power(e)[..., None]).flatten(-2)


def prepare(case, seed):
    c = dict(case)
    B, H, Hkv, Sq, Sk, D = (c[n] for n in ("B", "H", "Hkv", "Sq", "Sk", "D"))
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    s = dict(c, q=normal(B, H, Sq, D), k=normal(B, Hkv, Sk, D))
    if c["op"] == "select":
        # keys of a block have something in common: a slowly changing part under the noise
        nb = -(-Sk // c["block"])
        part = normal(B, Hkv, nb, D).repeat_interleave(c["block"], dim=2)[:, :, :Sk]
        s["k"] = s["k"] + part
        s["kv_len"], s["q_start"] = _positions(c, gen)
        s["start"] = s["means"] = None
        if Sq == 1:
            # the token's block has the mean of its earlier keys in the cache
            n = s["kv_len"] if s["kv_len"] is not None else torch.full((B,), Sk, device="cuda", dtype=torch.int32)
            s["means"] = _means(s["k"], c["block"], n - 1)
            s["start"] = n - 1
        return s
    s["v"] = normal(B, Hkv, Sk, D)
    if c["op"] in ("train", "attend"):
        s["kv_len"], s["q_start"] = _positions(c, gen)
        # neighbouring queries want much the same blocks: a score shared by 64 positions and
        # half as much of the query's own
        nb = -(-Sk // c["block"])
        shared = torch.randn(B, Hkv, -(-Sq // 64), nb, generator=gen, device="cuda")
        score = 0.5 * torch.randn(B, Hkv, Sq, nb, generator=gen, device="cuda")
        score += shared.repeat_interleave(64, dim=2)[:, :, :Sq]
        s["idx"] = _pick(score, _limits(s), c["block"], c["topk"])
        s["do"] = normal(B, H, Sq, D) if c["op"] == "train" else None
        return s
    if c["op"] == "ckpt":
        s["o"] = 0.2 * normal(B, H, Sq, D)
        return s
    s["do"] = normal(B, H, Sq, D)
    o, s["lse"] = _dense_forward(s["q"].float(), s["k"].float(), s["v"].float(), c["causal"])
    s["packed"] = [_pack(x) for x in (s.pop("q"), s.pop("k"), s.pop("v"), o.to(torch.bfloat16))]
    s["schedule"] = "sym_shift" if c["causal"] else "shift"
    return s


# ------------------------------------------------------------------ plain forms
def _means(k, block, n):
    """fp32 means of the blocks' keys below n [B] (0 where a block has none)."""
    B, Hkv, Sk, D = k.shape
    nb = -(-Sk // block)
    t = torch.arange(Sk, device=k.device)
    x = k.double().masked_fill((t >= n[:, None])[:, None, :, None], 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * block - Sk)).unflatten(2, (nb, block)).sum(3)
    first = torch.arange(nb, device=k.device) * block
    count = (n[:, None] - first).clamp(1, block)
    return (x / count[:, None, :, None]).float()


def _select(s):
    B, H, Hkv, Sk, block = s["B"], s["H"], s["Hkv"], s["Sk"], s["block"]
    n = s["kv_len"] if s["kv_len"] is not None else torch.full((B,), Sk, device="cuda", dtype=torch.int32)
    if s["means"] is None:
        means = _means(s["k"], block, n)
    else:
        # the block of the newest position alone
        at = (s["start"] // block).long()
        t = (at * block)[:, None] + torch.arange(block, device="cuda")
        there = t < n[:, None]
        rows = torch.arange(B, device="cuda")[:, None]
        x = s["k"][rows, :, t.clamp(max=Sk - 1)].double().masked_fill(~there[:, :, None, None], 0.0)
        means = s["means"]
        means[torch.arange(B, device="cuda"), :, at] = (x.sum(1) / there.sum(1)[:, None, None]).float()
    q = s["q"].double().unflatten(1, (Hkv, H // Hkv)).sum(2)
    return means, _pick(q @ means.double().transpose(-1, -2), _limits(s), block, s["topk"])


def _mask(s):
    """Which keys each query attends to, [B,Hkv,1,Sq,Sk]."""
    nb = -(-s["Sk"] // s["block"])
    on = torch.zeros(*s["idx"].shape[:3], nb + 1, dtype=torch.bool, device="cuda")
    on.scatter_(3, torch.where(s["idx"] < 0, nb, s["idx"]).long(), True)
    on = on[..., :nb].repeat_interleave(s["block"], dim=3)[..., : s["Sk"]]
    seen = torch.arange(s["Sk"], device="cuda") < _limits(s)[..., None]
    return (on & seen[:, None])[:, :, None]


def _sparse(s):
    Hkv, G, D = s["Hkv"], s["H"] // s["Hkv"], s["D"]
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().unflatten(1, (Hkv, G))
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    x = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~_mask(s), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1).flatten(1, 2)
    p.div_(total.masked_fill(total == 0, 1.0))
    o = p @ v
    out = [o.flatten(1, 2).to(torch.bfloat16), lse]
    if s["do"] is None:
        return out
    do = s["do"].float().unflatten(1, (Hkv, G))
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k).mul_(scale).flatten(1, 2)
    dk = (ds.transpose(-1, -2) @ q).sum(2).mul_(scale)
    return out + [dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)]


def _dense_forward(q, k, v, causal):
    Hkv = k.shape[1]
    q = q.unflatten(1, (Hkv, q.shape[1] // Hkv))
    x = (q @ k[:, :, None].transpose(-1, -2)).mul_(1.0 / math.sqrt(q.shape[-1]))
    if causal:
        x.masked_fill_(torch.ones(x.shape[-2:], dtype=torch.bool, device=x.device).triu_(1), -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return ((p @ v[:, :, None]) / total).flatten(1, 2), (top + total.log()).squeeze(-1).flatten(1, 2)


def _ckpt_backward(s):
    Hkv, G = s["Hkv"], s["H"] // s["Hkv"]
    scale = 1.0 / math.sqrt(s["D"])
    q, k, v, o = (_values(m, e) for m, e in s["packed"])
    q, o, do = (t.unflatten(1, (Hkv, G)) for t in (q, o, s["do"].float()))
    k, v = k[:, :, None], v[:, :, None]
    p = (q @ k.transpose(-1, -2)).mul_(scale).sub_(s["lse"].unflatten(1, (Hkv, G))[..., None]).exp_()
    if s["causal"]:
        p.tril_()
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k).mul_(scale).flatten(1, 2)
    dk = (ds.transpose(-1, -2) @ q).sum(2).mul_(scale)
    return [dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)]


def run(s):
    op = s["op"]
    if own:
        from persistent_sm_attn_b200 import binding as dash

        if op == "select":
            means = dash.dash_block_means(s["k"], s["block"], kv_len=s["kv_len"], start=s["start"], out=s["means"])
            idx = dash.dash_block_select(s["q"], means, s["Sk"], s["block"], s["topk"], causal=True, sink=1,
                                         local=1, kv_len=s["kv_len"], q_start=s["q_start"])
            return means, idx
        if op == "attend":
            return dash.dash_attn_sparse_fwd(s["q"], s["k"], s["v"], s["idx"], s["block"], causal=True,
                                             kv_len=s["kv_len"], q_start=s["q_start"])
        if op == "train":
            plan = dash.dash_sparse_plan(s["idx"], s["H"], s["Sk"], s["block"], causal=True,
                                         kv_len=s["kv_len"], q_start=s["q_start"])
            o, lse = dash.dash_attn_sparse_fwd(s["q"], s["k"], s["v"], s["idx"], s["block"], plan=plan)
            return o, lse, *dash.dash_attn_sparse_bwd(s["q"], s["k"], s["v"], o, s["do"], lse, plan)
        if op == "ckpt":
            packed = dash.dash_ckpt8_pack(s["q"], s["k"], s["v"], s["o"])
            return dash.dash_ckpt8_unpack(*packed)
        return dash.dash_attn_bwd_ckpt8(*s["packed"], s["do"], s["lse"], s["causal"], schedule=s["schedule"])
    if op == "select":
        return _select(s)
    if op in ("train", "attend"):
        return _sparse(s)
    if op == "ckpt":
        return [_values(*_pack(s[n])).to(torch.bfloat16) for n in ("q", "k", "v", "o")]
    return _ckpt_backward(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    B, H, Hkv, Sq, Sk, D = (c[n] for n in ("B", "H", "Hkv", "Sq", "Sk", "D"))
    rows, keys = B * H * Sq, B * Hkv * Sk
    if c["op"] == "ckpt":
        n = 2 * (rows + keys) * D
        return {"bytes": n * 2 * (2 + 1 + 1 / GROUP), "flops": 4 * n}
    if c["op"] == "ckpt_bwd":
        pairs = B * H * (Sq * (Sq + 1) // 2 if c["causal"] else Sq * Sk)
        return {"bytes": 2 * (rows + keys) * D * (1 + 1 / GROUP) + 2 * rows * D + 4 * rows + (rows + 2 * keys) * 2 * D,
                "flops": 10 * pairs * D}
    block, topk = c["block"], c["topk"]
    # mean length: a ragged batch's lengths are spread over the upper half
    length = (max(Sq, Sk // 2) + Sk) / 2 if c["ragged"] else Sk
    nb = -(-int(length) // block)
    if c["op"] == "select":
        read = B * Hkv * (min(block, length) if Sq == 1 else length) * D * 2
        seen = max(1.0, nb - (Sq / block - 1) / 2)  # visible blocks of a mean query
        return {"bytes": read + B * Hkv * nb * D * 4 + rows * D * 2 + 4 * B * Hkv * Sq * topk,
                "flops": 2 * B * Hkv * Sq * seen * D + rows * D}
    first = length - Sq  # position of query 0
    i = torch.arange(Sq, dtype=torch.float64) + first + 1
    picked = torch.minimum(i, (topk - 1) * block + (i - 1) % block + 1).sum().item()  # keys a head's queries attend to
    if Sq == 1:
        kv = 2 * B * Hkv * picked * D * 2
    else:
        kv = 2 * B * Hkv * length * D * 2
    io = kv + rows * (4 * D + 4) + 4 * B * Hkv * Sq * topk
    if c["op"] == "attend":
        return {"bytes": io, "flops": 4 * B * H * picked * D}
    return {"bytes": io + rows * 4 * D + 2 * keys * 2 * D, "flops": 14 * B * H * picked * D}


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_head(q, k, v, do, mask):
    """softmax(scale q k^T) v under `mask` for one K/V head's query heads [G,Sq,D], by
    automatic differentiation."""
    q, k, v = (t.double().requires_grad_(do is not None) for t in (q, k, v))
    x = torch.einsum("gid,jd->gij", q, k) / math.sqrt(q.shape[-1])
    some = mask.any(-1)
    x = torch.where(mask, x, -math.inf)
    x = torch.where(some[..., None], x, 0.0)
    lse = torch.where(some, torch.logsumexp(x, -1), -math.inf)
    o = torch.einsum("gij,jd->gid", torch.softmax(x, -1) * some[..., None], v)
    if do is None:
        return o, lse
    grads = torch.autograd.grad(o, (q, k, v), do.double())
    return (o.detach(), lse.detach(), *grads)


def _exact_attention(s):
    B, Hkv, G, Sk, block = s["B"], s["Hkv"], s["H"] // s["Hkv"], s["Sk"], s["block"]
    limit = _limits(s)
    t = torch.arange(Sk, device="cuda")
    got = []
    for b in range(B):
        for h in range(Hkv):
            chosen = torch.zeros(s["Sq"], -(-Sk // block) + 1, device="cuda")
            chosen.scatter_add_(1, s["idx"][b, h].long() + 1, torch.ones_like(s["idx"][b, h], dtype=torch.float32))
            mask = (chosen[:, 1:][:, t // block] > 0) & (t < limit[b][:, None])
            heads = slice(h * G, h * G + G)
            do = None if s["do"] is None else s["do"][b, heads]
            got.append(_exact_head(s["q"][b, heads], s["k"][b, h], s["v"][b, h], do, mask))
    parts = [torch.stack(x) for x in zip(*got)]
    out = [parts[0].reshape(B, s["H"], s["Sq"], -1), parts[1].reshape(B, s["H"], s["Sq"])]
    if s["do"] is not None:
        out += [parts[2].reshape(B, s["H"], s["Sq"], -1)] + [x.reshape(B, Hkv, Sk, -1) for x in parts[3:]]
    return out


def _exact_values(x):
    """What a checkpoint of x stands for: the nearest multiples of each group's step."""
    g = x.double().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    # the power of two at or below the largest element is that element without its fraction
    step = torch.where(top > 0, (top.view(torch.int64) >> 52 << 52).view(torch.float64) / 64, 1.0)
    return (torch.clamp(torch.round(g / step), -127, 127) * step).flatten(-2)


def _exact_ckpt_backward(s):
    B, H, Hkv, S, D = s["B"], s["H"], s["Hkv"], s["Sq"], s["D"]
    scale = 1.0 / math.sqrt(D)
    q, k, v, o = (m.double() * ((e.long() + 1023) << 52).view(torch.float64).repeat_interleave(GROUP, -1) for m, e in s["packed"])
    do, lse = s["do"].double(), s["lse"].double()
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        for h in range(H):
            g = h * Hkv // H
            p = torch.exp(scale * torch.einsum("id,jd->ij", q[b, h], k[b, g]) - lse[b, h, :, None])
            if s["causal"]:
                p = torch.tril(p)
            dp = torch.einsum("id,jd->ij", do[b, h], v[b, g])
            ds = scale * p * (dp - torch.einsum("id,id->i", do[b, h], o[b, h])[:, None])
            dq[b, h] = torch.einsum("ij,jd->id", ds, k[b, g])
            dk[b, g] += torch.einsum("ij,id->jd", ds, q[b, h])
            dv[b, g] += torch.einsum("ij,id->jd", p, do[b, h])
    return [dq, dk, dv]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("train", "attend"):
        return _exact_attention(s)
    if op == "ckpt":
        return [_exact_values(s[n]) for n in ("q", "k", "v", "o")]
    if op == "ckpt_bwd":
        return _exact_ckpt_backward(s)
    B, Hkv, Sk, block = s["B"], s["Hkv"], s["Sk"], s["block"]
    nb = -(-Sk // block)
    means = torch.zeros(B, Hkv, nb, s["D"], dtype=torch.float64, device="cuda")
    for b in range(B):
        n = Sk if s["kv_len"] is None else int(s["kv_len"][b])
        full = n // block
        means[b, :, :full] = s["k"][b, :, : full * block].double().unflatten(1, (full, block)).mean(2)
        if n % block:
            means[b, :, full] = s["k"][b, :, full * block : n].double().mean(1)
    return [means, None]
