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
