"""Block-sparse attention on the GPU: forward and backward against the 64-bit form, where they can
go wrong: odd lengths, heads that do not fill a tile, ragged batches, rows without keys, strides,
garbage past the sequences, repeated and unused picks, streams, graphs and determinism."""
import math

import pytest
import torch

from persistent_sm_attn_b200 import binding as dash
from tests import sparse_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def case(B, H, Hkv, Sq, Sk, D, block, topk, causal, ragged=False, seed=0, empty=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-Sk // block)
    c = dict(q=normal(gen, B, H, Sq, D), k=normal(gen, B, Hkv, Sk, D), v=normal(gen, B, Hkv, Sk, D),
             do=normal(gen, B, H, Sq, D), block=block, causal=causal, kv_len=None, q_start=None)
    # any block, any order, repeats, unused places and now and then a query without picks
    idx = torch.randint(-1, nb, (B, Hkv, Sq, topk), generator=gen, device="cuda", dtype=torch.int32)
    none = torch.rand(B, Hkv, Sq, generator=gen, device="cuda") < empty
    c["idx"] = torch.where(none[..., None], -1, idx)
    if ragged:
        c["kv_len"] = torch.randint(0, Sk + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        c["q_start"] = torch.randint(-2, max(1, Sk - Sq) + 1, (B,), generator=gen, device="cuda",
                                     dtype=torch.int32)
    return c


def ref_mask(c):
    B, _, Sq, _ = c["q"].shape
    Sk = c["k"].shape[2]
    lim = R.limits(B, Sq, Sk, c["causal"], c["kv_len"], c["q_start"], "cuda")
    return R.mask(c["idx"], Sk, c["block"], lim)


def run_fwd(c, **kw):
    return dash.dash_attn_sparse_fwd(c["q"], c["k"], c["v"], c["idx"], c["block"], c["causal"],
                                     c["kv_len"], c["q_start"], **kw)


def make_plan(c, **kw):
    return dash.dash_sparse_plan(c["idx"], c["q"].shape[1], c["k"].shape[2], c["block"], c["causal"],
                                 c["kv_len"], c["q_start"], **kw)


def check_fwd(c, o, lse, m=None, scale=None):
    m = ref_mask(c) if m is None else m
    want, wl, bound = R.forward(c["q"], c["k"], c["v"], m, scale)
    assert R.within(o, want, bound) <= 1.0
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (o[empty] == 0).all()
    # LSE: the score's fp32 error, and half a step of fp32 (2^-24) of values below 2^5
    assert (lse.double() - wl)[~empty].abs().max().item() <= R.SLACK if (~empty).any() else True
    return m


def check_bwd(c, o, lse, grads, m, scale=None):
    want, bounds = R.backward(c["q"], c["k"], c["v"], o, c["do"], lse, m, scale)
    for name, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        assert R.within(g, w, b) <= 1.0, name
    dead = ~m.any(2)
    assert (grads[1][dead] == 0).all() and (grads[2][dead] == 0).all()


SHAPES = [
    # B, H, Hkv, Sq, Sk, D, block, topk, causal, ragged
    (1, 1, 1, 1, 1, 64, 64, 1, True, False),
    (1, 2, 2, 64, 64, 128, 64, 1, True, False),
    (1, 2, 1, 65, 65, 128, 64, 2, True, False),
    (2, 4, 2, 200, 333, 64, 64, 3, True, True),
    (2, 4, 2, 200, 333, 128, 64, 3, True, True),
    (1, 3, 1, 130, 130, 128, 64, 2, True, False),     # 42 tokens a tile, two rows unused
    (1, 7, 1, 100, 700, 64, 128, 4, True, False),     # 18 tokens a tile
    (2, 16, 1, 33, 1000, 128, 128, 3, False, True),
    (1, 8, 8, 300, 300, 128, 256, 1, False, False),
    (1, 8, 8, 257, 511, 64, 64, 5, True, False),
    (1, 64, 1, 9, 129, 128, 64, 2, True, False),
    (1, 128, 1, 3, 200, 64, 64, 2, True, False),      # one token a tile
    (3, 2, 1, 1, 900, 128, 64, 4, True, True),        # single tokens
    (3, 32, 8, 1, 900, 64, 64, 16, True, True),
    (2, 4, 1, 5, 2000, 128, 128, 9, False, True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward_match_the_64_bit_form(shape):
    c = case(*shape[:9], ragged=shape[9], seed=hash(shape) % 1000)
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    m = check_fwd(c, o, lse)
    grads = dash.dash_attn_sparse_bwd(c["q"], c["k"], c["v"], o, c["do"], lse, plan)
    check_bwd(c, o, lse, grads, m)
    assert dash.dash_attn_sync_status() == 0


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_without_a_plan(shape):
    c = case(*shape[:9], ragged=shape[9], seed=hash(shape) % 1000 + 1)
    o, lse = run_fwd(c)
    check_fwd(c, o, lse)
    assert dash.dash_attn_sync_status() == 0


LARGE = [
    # more query tiles than SMs, lists of odd and even length, tiles without a unit
    (2, 8, 4, 3001, 3001, 128, 64, 5, True, False),
    (3, 4, 4, 6400, 6500, 64, 128, 3, True, True),
    (1, 3, 1, 9000, 300, 64, 64, 1, False, False),
    # more than 768 keys a query: dS with one part
    (1, 4, 2, 2500, 2500, 128, 64, 14, True, False),
    (1, 8, 8, 2100, 2000, 64, 128, 8, True, True),
]


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_many_tiles_of_a_cta(shape):
    c = case(*shape[:9], ragged=shape[9], seed=7)
    if shape[3] % 2 == 0:
        c["idx"][:, 1:, 1000:1700] = -1
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    grads = dash.dash_attn_sparse_bwd(c["q"], c["k"], c["v"], o, c["do"], lse, plan)
    assert dash.dash_attn_sync_status() == 0
    m = ref_mask(c)
    got = dict(o=o, lse=lse, dq=grads[0], dk=grads[1], dv=grads[2])
    G = shape[1] // shape[2]
    for b in range(shape[0]):  # the 64-bit form, a K/V head at a time
        for h in range(shape[2]):
            hs = slice(h * G, h * G + G)
            one = dict(q=c["q"][b:b + 1, hs], k=c["k"][b:b + 1, h:h + 1], v=c["v"][b:b + 1, h:h + 1],
                       do=c["do"][b:b + 1, hs])
            mm = m[b:b + 1, h:h + 1]
            check_fwd(one, o[b:b + 1, hs], lse[b:b + 1, hs], mm)
            check_bwd(one, o[b:b + 1, hs], lse[b:b + 1, hs],
                      (got["dq"][b:b + 1, hs], got["dk"][b:b + 1, h:h + 1], got["dv"][b:b + 1, h:h + 1]), mm)


TOKENS = [
    # B, H, Hkv, Sq, Sk, D, block, topk, causal, ragged
    (1, 1, 1, 1, 1, 64, 64, 1, True, False),
    (1, 32, 8, 1, 4096, 128, 64, 16, True, False),
    (5, 32, 8, 1, 3000, 128, 64, 16, True, True),
    (70, 16, 8, 1, 700, 64, 128, 3, True, True),      # a CTA for itself
    (2, 34, 2, 1, 777, 128, 64, 5, True, True),       # 17 heads: two groups of rows
    (1, 128, 1, 2, 300, 64, 64, 4, True, False),
    (3, 6, 2, 4, 1000, 128, 256, 2, False, True),
    (2, 4, 4, 3, 5000, 64, 64, 90, True, True),       # more picks than lanes, repeats across them
    (1, 7, 1, 1, 200, 128, 64, 1024, True, False),
]


@pytest.mark.parametrize("shape", TOKENS, ids=str)
def test_tokens_without_a_plan(shape):
    c = case(*shape[:9], ragged=shape[9], seed=hash(shape) % 1000)
    if shape[9]:  # what lies past the sequences may be anything
        for b in range(shape[0]):
            c["k"][b, :, int(c["kv_len"][b]):] = float("nan")
            c["v"][b, :, int(c["kv_len"][b]):] = float("inf")
    o, lse = run_fwd(c)
    check_fwd(c, o, lse)
    with_plan = run_fwd(c, plan=make_plan(c))
    check_fwd(c, *with_plan)
    again = run_fwd(c)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def grads_of(c, o, lse, plan, **kw):
    return dash.dash_attn_sparse_bwd(c["q"], c["k"], c["v"], o, c["do"], lse, plan, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_what_lies_past_the_sequences_is_not_used(D):
    c = case(3, 4, 2, 150, 500, D, 64, 4, True, ragged=True, seed=11)
    c["kv_len"] = torch.tensor([0, 77, 333], device="cuda", dtype=torch.int32)
    c["q_start"] = torch.tensor([-5, 100, 350], device="cuda", dtype=torch.int32)
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    want = grads_of(c, o, lse, plan)
    check_bwd(c, o, lse, want, check_fwd(c, o, lse))
    for b in range(3):
        n = int(c["kv_len"][b])
        c["k"][b, :, n:] = float("nan")
        c["v"][b, :, n:] = float("inf")
    o2, lse2 = run_fwd(c, plan=plan)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for x, y in zip(want, grads_of(c, o, lse, plan)):
        assert torch.equal(x, y)


def test_a_nan_stays_in_its_row():
    c = case(1, 4, 2, 100, 300, 64, 64, 3, True, seed=12, empty=0.0)
    c["idx"][..., 0] = 0
    plan = make_plan(c)
    o, _ = run_fwd(c, plan=plan)
    c["q"][0, 1, 40] = float("nan")
    o2, lse2 = run_fwd(c, plan=plan)
    bad = torch.zeros(1, 4, 100, dtype=torch.bool, device="cuda")
    bad[0, 1, 40] = True
    assert torch.isnan(o2[bad]).all() and torch.isnan(lse2[bad]).all()
    assert torch.equal(o2[~bad], o[~bad])
    c["q"], c["idx"], c["do"] = c["q"][:, :, 40:41], c["idx"][:, :, 40:41], None
    o3, lse3 = dash.dash_attn_sparse_fwd(c["q"].contiguous(), c["k"], c["v"], c["idx"].contiguous(), 64,
                                         q_start=torch.tensor([240], device="cuda", dtype=torch.int32))
    assert torch.isnan(o3[0, 1]).all() and torch.isfinite(o3[0, [0, 2, 3]].float()).all()


@pytest.mark.parametrize("Sq", [1, 130])
def test_strided_inputs(Sq):
    c = case(2, 6, 3, Sq, 400, 64, 64, 4, True, seed=13)
    o, lse = run_fwd(c)
    t = dict(c)
    for n in ("q", "k", "v", "do"):  # [B,S,H,D] in memory, and rows of a wider buffer
        wide = torch.full((*c[n].transpose(1, 2).shape[:3], 72), float("nan"), device="cuda",
                          dtype=torch.bfloat16)
        wide[..., :64] = c[n].transpose(1, 2)
        t[n] = wide[..., :64].transpose(1, 2)
        assert torch.equal(t[n], c[n]) and not t[n].is_contiguous()
    o2, lse2 = run_fwd(t)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    plan = make_plan(c)
    for x, y in zip(grads_of(c, o, lse, plan), grads_of(t, o, lse, plan)):
        assert torch.equal(x, y)
    with pytest.raises(ValueError, match="strides"):
        run_fwd(dict(c, k=c["k"][:, :1].expand(2, 3, 400, 64)))
    with pytest.raises(ValueError, match="last dimension"):
        run_fwd(dict(c, q=c["q"].transpose(2, 3).contiguous().transpose(2, 3) if Sq > 1
                     else c["q"].new_zeros(2, 6, 1, 128)[..., ::2]))
    with pytest.raises(ValueError, match="aligned"):
        run_fwd(dict(c, v=c["v"].new_zeros(2 * 3 * 400 * 64 + 1)[1:].view(2, 3, 400, 64)))


def test_a_selection_counts_each_block_once_and_in_any_order():
    c = case(1, 4, 2, 190, 640, 64, 64, 4, True, seed=14, empty=0.0)
    perm = torch.randperm(4, device="cuda")
    more = torch.cat([c["idx"][..., perm], c["idx"], torch.full_like(c["idx"], 99),
                      torch.full_like(c["idx"], -7)], -1).contiguous()
    o, lse = run_fwd(c, plan=make_plan(c))
    o2, lse2 = run_fwd(dict(c, idx=more), plan=make_plan(dict(c, idx=more)))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    few = dict(c, q=c["q"][:, :, -3:].contiguous(), idx=more[:, :, -3:].contiguous())  # no plan
    check_fwd(few, *run_fwd(few))


def test_results_are_reproducible():
    c = case(2, 8, 2, 700, 1500, 128, 64, 6, True, seed=15)
    runs = []
    for _ in range(3):
        plan = make_plan(c)
        o, lse = run_fwd(c, plan=plan)
        runs.append((o, lse, *grads_of(c, o, lse, plan)))
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert torch.equal(x, y)


def test_empty_batches_and_no_queries():
    for B, Sq in ((0, 5), (2, 0)):
        c = case(2, 4, 2, 5, 100, 64, 64, 2, True, seed=16)
        for n in ("q", "do"):
            c[n] = c[n][:B, :, :Sq].contiguous()
        c["k"], c["v"] = c["k"][:B].contiguous(), c["v"][:B].contiguous()
        c["idx"] = c["idx"][:B, :, :Sq].contiguous()
        plan = make_plan(c)
        o, lse = run_fwd(c, plan=plan)
        assert o.shape == c["q"].shape and lse.shape == (B, 4, Sq)
        assert run_fwd(c)[0].shape == o.shape
        dq, dk, dv = grads_of(c, o, lse, plan)
        assert dq.shape == c["q"].shape and (dk == 0).all() and (dv == 0).all()
    assert dash.dash_attn_sync_status() == 0


def test_refusals():
    c = case(1, 4, 2, 8, 256, 64, 64, 2, True, seed=17)
    plan = make_plan(c)
    with pytest.raises(ValueError, match="the plan is for"):
        dash.dash_attn_sparse_fwd(c["q"][:, :, :4].contiguous(), c["k"], c["v"], None, 64, plan=plan)
    with pytest.raises(ValueError, match="idx"):
        run_fwd(dict(c, idx=c["idx"][:, :, :4].contiguous()))
    with pytest.raises(ValueError, match="idx"):
        run_fwd(dict(c, idx=c["idx"].long()))
    with pytest.raises(ValueError, match="kv_len"):
        run_fwd(dict(c, kv_len=torch.zeros(2, device="cuda", dtype=torch.int32)))
    with pytest.raises(ValueError, match="block"):
        run_fwd(dict(c, block=100))
    with pytest.raises(ValueError, match="v has shape"):
        run_fwd(dict(c, v=c["v"][:, :1].contiguous()))
    with pytest.raises(ValueError, match="out"):
        run_fwd(c, out=torch.empty_like(c["k"]))
    with pytest.raises(dash.DashError):
        run_fwd(c, scale=-1.0)
    with pytest.raises(dash.DashError):
        run_fwd(dict(c, q=c["q"][:, :3].contiguous()))


def test_scale_and_given_outputs():
    c = case(1, 4, 2, 200, 300, 128, 64, 3, False, seed=18)
    out, lse = torch.empty_like(c["q"]), torch.empty(1, 4, 200, device="cuda")
    o, l = run_fwd(c, scale=0.3, plan=make_plan(c), out=out, lse=lse)
    assert o is out and l is lse
    # scores are 0.3 sqrt(128) = 3.4 times those of the default scale: so is their fp32 error
    want, wl, bound = R.forward(c["q"], c["k"], c["v"], ref_mask(c), 0.3)
    assert R.within(o, want, bound * (R.HALF + 3.4 * R.SLACK) / (R.HALF + R.SLACK)) <= 1.0


def test_offsets_past_32_bits():
    # a cache of two sequences 2^31 elements apart, another row stride than D
    row, far = 72, 2 ** 31 + 8
    kb = torch.zeros(far + 600 * row, device="cuda", dtype=torch.bfloat16)
    vb = torch.zeros_like(kb)
    c = case(2, 4, 1, 40, 600, 64, 64, 3, True, seed=19)
    k = kb.as_strided((2, 1, 600, 64), (far, 600 * row, row, 1))
    v = vb.as_strided((2, 1, 600, 64), (far, 600 * row, row, 1))
    k.copy_(c["k"])
    v.copy_(c["v"])
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    f = dict(c, k=k, v=v)
    o2, lse2 = run_fwd(f, plan=plan)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for x, y in zip(grads_of(c, o, lse, plan), grads_of(f, o, lse, plan)):
        assert torch.equal(x, y)
    one = lambda d: dict(d, q=d["q"][:, :, -1:].contiguous(), idx=d["idx"][:, :, -1:].contiguous())
    for x, y in zip(run_fwd(one(c)), run_fwd(one(f))):
        assert torch.equal(x, y)
    assert torch.equal(dash.dash_block_means(k, 64), dash.dash_block_means(c["k"], 64))


def layer_step(q, k, v, do, n, start, topk=4, stream=None):
    """A training step of a sparse layer from checkpoints: select, attend, pack, go back."""
    Sk = k.shape[2]
    means = dash.dash_block_means(k, 64, n, stream=stream)
    idx = dash.dash_block_select(q, means, Sk, 64, topk, kv_len=n, q_start=start, stream=stream)
    plan = dash.dash_sparse_plan(idx, q.shape[1], Sk, 64, kv_len=n, q_start=start, stream=stream)
    o, lse = dash.dash_attn_sparse_fwd(q, k, v, idx, 64, plan=plan, stream=stream)
    packed = dash.dash_ckpt8_pack(q, k, v, o, stream=stream)
    return (idx, o, lse, *dash.dash_attn_sparse_bwd_ckpt8(*packed, do, lse, plan, stream=stream))


def step_inputs(seed, ragged=True):
    c = case(2, 4, 2, 300, 300, 64, 64, 4, True, seed=seed)
    n = torch.tensor([300, 211], device="cuda", dtype=torch.int32) if ragged else None
    return c["q"], c["k"], c["v"], c["do"], n, (n - n if ragged else None)


def test_a_step_from_selection_to_gradients():
    q, k, v, do, n, start = step_inputs(20)
    idx, o, lse, *grads = layer_step(q, k, v, do, n, start)
    means = dash.dash_block_means(k, 64, n)
    assert torch.equal(idx.cpu(), R.select(q, means, 300, 64, 4, True, 1, 1, n, start))
    c = dict(q=q, k=k, v=v, do=do, idx=idx, block=64, causal=True, kv_len=n, q_start=start)
    m = check_fwd(c, o, lse)
    vals = [R.ckpt_values(*R.ckpt_pack(x)).to(torch.bfloat16) for x in (q, k, v, o)]
    want, bounds = R.backward(*vals, do, lse, m)
    for g, w, b in zip(grads, want, bounds):
        assert R.within(g, w, b) <= 1.0


def test_a_cache_that_grows_token_by_token():
    B, H, Hkv, D, block, cap = 3, 8, 2, 64, 64, 400
    gen = torch.Generator(device="cuda").manual_seed(21)
    k, v = normal(gen, B, Hkv, cap, D), normal(gen, B, Hkv, cap, D)
    n = torch.tensor([1, 127, 383], device="cuda", dtype=torch.int32)
    means = dash.dash_block_means(k, block, n)
    for step in range(4):
        n = n + 1
        q = normal(gen, B, H, 1, D)
        dash.dash_block_means(k, block, n, start=n - 1, out=means)
        assert torch.equal(means, dash.dash_block_means(k, block, n))
        idx = dash.dash_block_select(q, means, cap, block, 3, kv_len=n, q_start=n - 1)
        assert torch.equal(idx.cpu(), R.select(q, means, cap, block, 3, True, 1, 1, n, n - 1))
        c = dict(q=q, k=k, v=v, idx=idx, block=block, causal=True, kv_len=n, q_start=n - 1)
        check_fwd(c, *run_fwd(c))


def test_steps_on_two_streams_and_in_graphs():
    a, b = step_inputs(22), step_inputs(23)
    want = [layer_step(*x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [layer_step(*x, stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    # two graphs, replayed at the same time on two streams, with inputs that change
    held = [[x.clone() if x is not None else None for x in a] for _ in range(2)]
    graphs, outs = [], []
    for h in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer_step(*h))
        graphs.append(g)
    for first, second in ((a, b), (b, a)):
        for h, x in zip(held, (first, second)):
            for dst, src in zip(h, x):
                dst.copy_(src)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, x in zip(outs, (first, second)):
            w = want[0] if x is a else want[1]
            assert all(torch.equal(p, q) for p, q in zip(o, w))
    for s in streams:
        assert dash.dash_attn_sync_status(s) == 0


def test_gradients_against_differences():
    # f = sum(O * dO) along a direction: (f(x + h d) - f(x - h d)) / 2h in 64 bits against <grad, d>
    c = case(1, 4, 2, 70, 200, 64, 64, 2, True, seed=24, empty=0.1)
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    m = ref_mask(c)
    grads = grads_of(c, o, lse, plan)
    _, bounds = R.backward(c["q"], c["k"], c["v"], o, c["do"], lse, m)
    # delta comes from the rounded O: off by HALF sum |dO o O| a row, times the formula's terms
    exact = [t.double() for t in (c["q"], c["k"], c["v"])]
    f = lambda q, k, v: (R.forward(q, k, v, m)[0] * c["do"].double()).sum()
    qd, kd, vd = exact
    G = 2
    g4 = lambda t: t.double().unflatten(1, (2, G))
    x = torch.einsum("bhgid,bhjd->bhgij", g4(qd), kd) / 8
    p = torch.where(m[:, :, None], torch.exp(x - g4(lse)[..., None]), 0.0)
    off = p * R.HALF * (g4(c["do"]) * g4(o)).abs().sum(-1, keepdim=True)
    extra = (torch.einsum("bhgij,bhjd->bhgid", off, kd.abs()).flatten(1, 2) / 8,
             torch.einsum("bhgij,bhgid->bhjd", off, g4(qd).abs()) / 8, 0.0)
    gen = torch.Generator(device="cuda").manual_seed(25)
    for i in range(3):
        d = torch.randn(exact[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = list(exact), list(exact)
        up[i], down[i] = exact[i] + h * d, exact[i] - h * d
        diff = (f(*up) - f(*down)) / (2 * h)
        got = (grads[i].double() * d).sum()
        bound = ((bounds[i] + extra[i]) * d.abs()).sum()
        assert (got - diff).abs() <= bound + 1e-6 * diff.abs() + 1e-6


FIRST_USE = """
import torch
from persistent_sm_attn_b200 import binding as dash
g = torch.Generator(device="cuda").manual_seed(1)
mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
q, k, v, do = mk(1, 4, 300, 64), mk(1, 2, 300, 64), mk(1, 2, 300, 64), mk(1, 4, 300, 64)
torch.cuda.synchronize()

def step():
    means = dash.dash_block_means(k, 64)
    idx = dash.dash_block_select(q, means, 300, 64, 3)
    plan = dash.dash_sparse_plan(idx, 4, 300, 64)
    o, lse = dash.dash_attn_sparse_fwd(q, k, v, idx, 64, plan=plan)
    packed = dash.dash_ckpt8_pack(q, k, v, o)
    grads = dash.dash_attn_sparse_bwd_ckpt8(*packed, do, lse, plan)
    one = q[:, :, -1:].contiguous()
    last = dash.dash_block_select(one, means, 300, 64, 3)
    return (o, lse, *grads, *dash.dash_attn_sparse_fwd(one, k, v, last, 64))

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(held, step()):
    assert torch.equal(a, b)
assert dash.dash_attn_sync_status() == 0
print("same")
"""


def test_the_first_use_may_be_captured():
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", FIRST_USE], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and "same" in out.stdout, out.stderr[-2000:]


@pytest.mark.parametrize("Sq", [1, 140])
def test_a_block_longer_than_the_sequence(Sq):
    # the same as a block of the sequence's length, in time as well
    a = case(2, 4, 2, Sq, 200, 64, 256, 2, True, ragged=True, seed=31)
    b = dict(a, block=1 << 30)
    results = []
    for c in (a, b):
        means = dash.dash_block_means(c["k"], c["block"], kv_len=c["kv_len"])
        idx = dash.dash_block_select(c["q"], means, 200, c["block"], 2, kv_len=c["kv_len"],
                                     q_start=c["q_start"])
        plan = make_plan(c)
        o, lse = run_fwd(c, plan=plan)
        results.append((means, idx, *run_fwd(c), o, lse,
                        *dash.dash_attn_sparse_bwd(c["q"], c["k"], c["v"], o, c["do"], lse, plan)))
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_the_forward_and_its_plan_agree():
    c = case(2, 4, 2, 190, 640, 64, 64, 4, False, seed=41)
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    for call in (lambda: dash.dash_attn_sparse_fwd(c["q"], c["k"], c["v"], c["idx"], 64, plan=plan),
                 lambda: dash.dash_attn_sparse_fwd(c["q"], c["k"], c["v"], None, 64, plan=plan)):
        x, y = call()  # the mask is the plan's
        assert torch.equal(x, o) and torch.equal(y, lse)
    check_fwd(c, o, lse)
    full = dash.dash_attn_sparse_fwd(c["q"], c["k"], c["v"], c["idx"], 64)  # causal without a plan
    check_fwd(dict(c, causal=True), *full)
    n = torch.full((2,), 640, device="cuda", dtype=torch.int32)
    for bad in (dict(c, causal=True), dict(c, block=128), dict(c, idx=c["idx"][..., :3].contiguous()),
                dict(c, kv_len=n), dict(c, q_start=n)):
        with pytest.raises(ValueError, match="the plan"):
            run_fwd(bad, plan=plan)


def test_no_queries_before_a_strided_cache():
    c = case(1, 4, 2, 0, 300, 64, 64, 2, True, seed=42)
    wide = torch.zeros(1, 300, 2, 72, device="cuda", dtype=torch.bfloat16)
    c["k"] = c["v"] = wide[..., :64].transpose(1, 2)
    o, lse = run_fwd(c)
    assert o.shape == (1, 4, 0, 64) and lse.shape == (1, 4, 0)
    plan = make_plan(c)
    dq, dk, dv = grads_of(c, *run_fwd(c, plan=plan), plan)
    assert dq.shape == o.shape and (dk == 0).all() and (dv == 0).all()


def test_no_query_heads():
    c = case(2, 2, 2, 5, 100, 64, 64, 2, True, seed=43)
    c["q"], c["do"] = (c[n][:, :0].contiguous() for n in ("q", "do"))
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    assert o.shape == (2, 0, 5, 64) and lse.shape == (2, 0, 5)
    assert run_fwd(c)[0].shape == o.shape
    held = torch.full_like(c["k"], float("nan")), torch.full_like(c["v"], float("nan"))
    dq, dk, dv = grads_of(c, o, lse, plan, dk=held[0], dv=held[1])
    assert dq.shape == o.shape and dk is held[0] and (dk == 0).all() and (dv == 0).all()
    with pytest.raises(dash.DashError):
        dash.dash_block_select(c["q"], dash.dash_block_means(c["k"], 64), 100, 64, 2)


def test_a_scale_of_zero_is_refused():
    c = case(1, 4, 2, 200, 256, 64, 64, 2, True, seed=44)
    plan = make_plan(c)
    o, lse = run_fwd(c, plan=plan)
    few = dict(c, q=c["q"][:, :, :2].contiguous(), idx=c["idx"][:, :, :2].contiguous())
    for call in (lambda s: run_fwd(c, scale=s), lambda s: run_fwd(few, scale=s),
                 lambda s: run_fwd(c, plan=plan, scale=s), lambda s: grads_of(c, o, lse, plan, scale=s)):
        for scale in (0.0, 1e-50):
            with pytest.raises(ValueError, match="scale"):
                call(scale)
        for scale in (-1.0, float("nan"), float("inf"), 1e39):
            with pytest.raises(dash.DashError):
                call(scale)


def test_the_current_stream_by_the_public_call(monkeypatch):
    c = case(2, 4, 2, 70, 200, 64, 64, 2, True, seed=45)
    o, lse = run_fwd(c)
    torch.cuda.synchronize()
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with dash._Launch(c["q"].device, None) as handle:
            assert handle == side.cuda_stream
        o2, lse2 = run_fwd(c)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
