"""Block means and block selection on the GPU against the definition, block by block and query by
query: the picks have to be equal."""
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


def inputs(B, H, Hkv, Sq, Sk, D, ragged, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k = normal(gen, B, H, Sq, D), normal(gen, B, Hkv, Sk, D)
    n = s = None
    if ragged:
        n = torch.randint(0, Sk + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s = torch.randint(-2, max(1, Sk - Sq) + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    return q, k, n, s


@pytest.mark.parametrize("B,Hkv,Sk,D,block,ragged", [
    (1, 1, 1, 64, 64, False), (2, 3, 65, 128, 64, True), (1, 2, 1000, 64, 128, False),
    (3, 1, 777, 128, 256, True), (2, 2, 640, 128, 320, True)])
def test_means(B, Hkv, Sk, D, block, ragged):
    _, k, n, _ = inputs(B, Hkv, Hkv, 1, Sk, D, ragged, 1)
    got = dash.dash_block_means(k, block, n)
    want = R.means(k, block, n)
    # the sum is exact, the quotient rounds twice (fp64, fp32): half a step of fp32 and a little
    assert (got.double() - want).abs().le(want.abs() * 2.0 ** -23.9).all()


def test_means_update_leaves_the_other_blocks():
    _, k, _, _ = inputs(3, 2, 2, 1, 500, 64, False, 2)
    n = torch.tensor([500, 130, 64], device="cuda", dtype=torch.int32)
    start = torch.tensor([300, 129, 64], device="cuda", dtype=torch.int32)
    means = torch.full((3, 2, 8, 64), 7.0, device="cuda")
    out = dash.dash_block_means(k, 64, n, start, out=means)
    assert out is means
    want = dash.dash_block_means(k, 64, n)
    touched = {0: range(4, 8), 1: range(2, 3), 2: range(0)}
    for b in range(3):
        for j in range(8):
            same = means[b, :, j] == (want[b, :, j] if j in touched[b] else 7.0)
            assert same.all(), (b, j)


def test_means_ignore_what_lies_past_the_sequence_and_take_strides():
    _, k, _, _ = inputs(2, 3, 3, 1, 200, 64, False, 3)
    n = torch.tensor([70, 199], device="cuda", dtype=torch.int32)
    bad = k.clone()
    bad[0, :, 70:] = float("nan")
    bad[1, :, 199:] = float("inf")
    view = bad.transpose(1, 2).contiguous().transpose(1, 2)  # [B,S,H,D] in memory
    assert not view.is_contiguous()
    assert torch.equal(dash.dash_block_means(view, 64, n), dash.dash_block_means(k, 64, n))


SHAPES = [
    # B, H, Hkv, Sq, Sk, D, block, topk, causal, sink, local, ragged
    (1, 1, 1, 1, 1, 64, 64, 1, True, 1, 0, False),
    (1, 4, 2, 130, 130, 64, 64, 2, True, 1, 1, False),
    (2, 4, 4, 77, 1500, 128, 64, 5, True, 1, 2, True),
    (2, 6, 2, 33, 3000, 128, 64, 16, True, 0, 0, True),
    (1, 8, 1, 40, 2500, 64, 128, 30, False, 2, 2, True),
    (3, 7, 1, 1, 5000, 64, 64, 8, True, 1, 1, True),
    (1, 2, 1, 3, 70000, 64, 64, 9, True, 1, 1, False),
    (2, 4, 2, 70, 20000, 64, 64, 12, True, 1, 1, True),   # 313 blocks
    (1, 2, 1, 40, 40000, 128, 64, 20, True, 1, 1, False),   # 625
    (1, 2, 1, 33, 70000, 64, 64, 9, True, 1, 1, False),   # 1094
    (1, 1, 1, 20, 262144, 64, 64, 5, True, 1, 1, False),  # 4096
    (1, 3, 1, 64, 5000, 64, 64, 2, True, 1, 1, False),    # every place is forced
    (1, 2, 1, 5, 100, 128, 256, 4, True, 1, 1, False),    # fewer blocks than places
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_select_matches_the_definition(shape):
    B, H, Hkv, Sq, Sk, D, block, topk, causal, sink, local, ragged = shape
    q, k, n, s = inputs(B, H, Hkv, Sq, Sk, D, ragged, sum(shape))
    means = dash.dash_block_means(k, block, n)
    got = dash.dash_block_select(q, means, Sk, block, topk, causal, sink, local, n, s)
    want = R.select(q, means, Sk, block, topk, causal, sink, local, n, s)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("Sq", [1, 300])
def test_equal_scores_go_to_the_lowest_block_and_near_ones_are_told_apart(Sq):
    # all blocks alike but for one bit of one fp32 mean: the fp32 score would not show it
    q = torch.ones(1, 2, Sq, 64, device="cuda", dtype=torch.bfloat16)
    means = torch.full((1, 1, 40, 64), 1.0, device="cuda")
    got = dash.dash_block_select(q, means, 40 * 64, 64, 6, False, 1, 1)
    assert (got.cpu() == torch.tensor([0, 1, 2, 3, 4, 39], dtype=torch.int32)).all()
    means[0, 0, 17, 5] = 1.0 + 2.0 ** -23
    means[0, 0, 30, 9] = 1.0 - 2.0 ** -24
    means[0, 0, 2, 9] = 1.0 - 2.0 ** -24
    got = dash.dash_block_select(q, means, 40 * 64, 64, 6, False, 1, 1)
    assert (got.cpu() == torch.tensor([0, 1, 3, 4, 17, 39], dtype=torch.int32)).all()


@pytest.mark.parametrize("Sq", [1, 17])
def test_zeros_of_either_sign_tie_and_nan_ranks_last(Sq):
    q = torch.ones(1, 1, Sq, 64, device="cuda", dtype=torch.bfloat16)
    means = torch.zeros(1, 1, 6, 64, device="cuda")
    means[0, 0, 0] = -0.0
    means[0, 0, 1] = float("nan")
    means[0, 0, 2] = float("-inf")
    means[0, 0, 5] = float("inf")
    pick = lambda n: dash.dash_block_select(q, means, 6 * 64, 64, n, False, 0, 0)[0, 0, -1].tolist()
    assert pick(1) == [5] and pick(2) == [0, 5] and pick(4) == [0, 3, 4, 5]
    assert pick(5) == [0, 2, 3, 4, 5] and pick(6) == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("Sq", [2, 100])
def test_zero_queries_and_large_values(Sq):
    q, k, _, _ = inputs(1, 2, 1, Sq, 2000, 64, False, 6)
    q[:, :, ::2] = 0  # a padding row: every block ties
    q[:, :, 1] *= 1e30
    k[:, :, 300:400] *= 1e8
    means = dash.dash_block_means(k, 64)
    got = dash.dash_block_select(q, means, 2000, 64, 5, False, 1, 1)
    assert torch.equal(got.cpu(), R.select(q, means, 2000, 64, 5, False, 1, 1))
    assert (got[0, 0, 0].cpu() == torch.tensor([0, 1, 2, 3, 31], dtype=torch.int32)).all()


def test_select_takes_strided_queries():
    q, k, _, _ = inputs(2, 4, 2, 50, 900, 64, False, 5)
    means = dash.dash_block_means(k, 64)
    view = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert not view.is_contiguous()
    assert torch.equal(dash.dash_block_select(view, means, 900, 64, 4),
                       dash.dash_block_select(q, means, 900, 64, 4))


@pytest.mark.parametrize("Sq", [1, 40])
@pytest.mark.parametrize("far", [1e3, 1e6])
def test_heads_that_cancel(Sq, far):
    # the heads' sum in fp32 would lose what decides: 1000 + x - 1000 keeps few bits of x
    q, k, _, _ = inputs(1, 4, 1, Sq, 3000, 64, False, 7)
    q[:, 0], q[:, 2] = far, -far
    q[:, 1] *= 1e-3
    q[:, 3] *= 1e-3
    means = dash.dash_block_means(k, 64)
    got = dash.dash_block_select(q, means, 3000, 64, 9, False, 1, 1)
    assert torch.equal(got.cpu(), R.select(q, means, 3000, 64, 9, False, 1, 1))


def select_into_guarded(q, means, Sk, topk):
    """The picks, written into the middle of a larger buffer of which nothing else may change."""
    B, _, Sq, _ = q.shape
    Hkv = means.shape[1]
    n, pad = B * Hkv * Sq * topk, 4096
    buf = torch.full((n + 2 * pad,), -77, device="cuda", dtype=torch.int32)
    out = buf[pad:pad + n].view(B, Hkv, Sq, topk)
    dash.dash_block_select(q, means, Sk, 64, topk, False, 1, 1, out=out)
    assert (buf[:pad] == -77).all() and (buf[pad + n:] == -77).all()
    return out.cpu()


# powers of ten that bf16 holds: an fp32 square is 0 from 1e-23 on, a bf16 subnormal from 1e-38
@pytest.mark.parametrize("Sq", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qs,ks", [(1e-12, 1.0), (1e-17, 1e-6), (1e-20, 1.0), (1e-23, 1.0), (1e-25, 1.0),
                                   (1e-30, 1.0), (1e-38, 1.0), (1.0, 1e-17), (1.0, 1e-23), (1.0, 1e-25),
                                   (1.0, 1e-38), (1e-25, 1e-25), (1e-19, 1e-19), (1e-30, 1e25)])
def test_tiny_operands(Sq, D, qs, ks):
    q, k, _, _ = inputs(1, 2, 1, Sq, 40 * 64, D, False, 8)
    q, k = (q.double() * qs).to(torch.bfloat16), (k.double() * ks).to(torch.bfloat16)
    means = dash.dash_block_means(k, 64)
    want = R.select(q, means, 40 * 64, 64, 6, False, 1, 1)
    assert torch.equal(select_into_guarded(q, means, 40 * 64, 6), want)


def test_tiny_queries_and_blocks_beside_ordinary_ones():
    q, k, _, _ = inputs(2, 3, 1, 100, 3000, 64, False, 9)
    q[0, :, ::3] *= 1e-25
    q[1, :, 1::3] *= 1e-38
    k[:, :, 640:1280] *= 1e-25
    k[1, :, 2000:] = 0
    means = dash.dash_block_means(k, 64)
    assert torch.equal(select_into_guarded(q, means, 3000, 9), R.select(q, means, 3000, 64, 9, False, 1, 1))
    for i in (0, 1, 3):
        one = q[:, :, i:i + 1].contiguous()
        assert torch.equal(select_into_guarded(one, means, 3000, 9),
                           R.select(one, means, 3000, 64, 9, False, 1, 1))
