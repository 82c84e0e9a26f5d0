"""Waits that run out in the middle of a launch, loads in flight: the status says so, the context
stays usable and the next call is right.  The fault is made on the host (a first dQ contributor
that never arrives, or a limit shorter than any wait of a working launch)."""
import pytest
import torch

from persistent_sm_attn_b200 import binding as dash
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

TIMEOUT = 4


@pytest.fixture(autouse=True)
def limits():
    G.need_cuda()
    yield
    dash.dash_inject_fault(0)
    dash.dash_set_spin_limit_us(0)
    dash.dash_set_dq_chain_mode(0)


# D, causal, schedule, red chains, limit in us.  Each CTA has many more tiles than stages when the
# limit strikes, so its producers are at work then.
CASES = [(64, False, "shift", 2, 1), (64, True, "descending", 1, 50), (64, True, "sym_shift", 0, 1),
         (128, False, "shift", 1, 50), (128, True, "descending", 1, 1), (128, True, "sym_shift", 2, 200),
         (64, False, "shift_pairs", 0, 1), (128, False, "shift_pairs", 0, 50),
         (128, True, "sym_shift_pairs", 0, 1), (64, True, "sym_shift_pairs", 0, 200)]


@pytest.mark.parametrize("D,causal,sched,red,limit", CASES)
def test_a_backward_that_runs_out_while_loads_are_in_flight(D, causal, sched, red, limit):
    case = G.make_case(1, 24, 2048, D, causal, seed=41)
    args = [case[n] for n in ("q", "k", "v", "o", "do", "lse")]
    dash.dash_set_dq_chain_mode(red)
    want = G.bwd(case, sched)
    pairs = sched.endswith("pairs")  # their tables take no planted fault: the limit alone
    for _ in range(4):
        dash.dash_set_spin_limit_us(limit)
        dash.dash_inject_fault(0 if pairs else 1)
        dash.dash_attn_bwd(*args, causal, sched)
        status = dash.dash_attn_sync_status()
        assert status == TIMEOUT or (pairs and status == 0)
        dash.dash_set_spin_limit_us(0)
        for a, b in zip(G.bwd(case, sched), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("D,causal", [(64, True), (128, False)])
def test_a_forward_with_the_shortest_limit(D, causal):
    case = G.make_case(2, 16, 2048, D, causal, seed=43)
    for _ in range(4):
        dash.dash_set_spin_limit_us(1)
        dash.dash_attn_fwd(case["q"], case["k"], case["v"], causal)
        assert dash.dash_attn_sync_status() in (0, TIMEOUT)  # whether a wait is that long is the GPU's
        dash.dash_set_spin_limit_us(0)
        o, lse = dash.dash_attn_fwd(case["q"], case["k"], case["v"], causal)
        assert dash.dash_attn_sync_status() == 0
        assert torch.equal(o, case["o"]) and torch.equal(lse, case["lse"])


def sparse_case(D, Sq=3000, H=6, Hkv=3, topk=14, seed=44):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda h: torch.randn(2, h, Sq, D, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v, do = mk(H), mk(Hkv), mk(Hkv), mk(H)
    idx = torch.randint(0, -(-Sq // 64), (2, Hkv, Sq, topk), generator=gen, device="cuda", dtype=torch.int32)
    return q, k, v, do, idx


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("limit", [1, 2000])
def test_block_sparse_calls_that_run_out(D, limit):
    q, k, v, do, idx = sparse_case(D)
    plan = dash.dash_sparse_plan(idx, 6, 3000, 64)
    forward = lambda: dash.dash_attn_sparse_fwd(q, k, v, idx, 64, plan=plan)
    o, lse = forward()
    backward = lambda: dash.dash_attn_sparse_bwd(q, k, v, o, do, lse, plan)
    want = backward()
    assert dash.dash_attn_sync_status() == 0
    side = torch.cuda.Stream()
    for call, right in ((forward, (o, lse)), (backward, want)) * 2:
        dash.dash_set_spin_limit_us(limit)
        dash.dash_inject_fault(2)
        call()
        # the stream that ran out reports it once; another one has nothing to report
        assert dash.dash_attn_sync_status(side) == 0
        assert dash.dash_attn_sync_status() == TIMEOUT
        assert dash.dash_attn_sync_status() == 0
        dash.dash_set_spin_limit_us(0)
        for a, b in zip(call(), right):
            assert torch.equal(a, b)
        assert dash.dash_attn_sync_status() == 0


def test_a_cancelled_fault_is_not_taken():
    q, k, v, _, idx = sparse_case(64, Sq=500)
    dash.dash_inject_fault(2)
    dash.dash_inject_fault(0)
    dash.dash_attn_sparse_fwd(q, k, v, idx, 64, plan=dash.dash_sparse_plan(idx, 6, 500, 64))
    assert dash.dash_attn_sync_status() == 0


def test_dense_and_block_sparse_timeouts_are_both_reported():
    q, k, v, _, idx = sparse_case(64)
    plan = dash.dash_sparse_plan(idx, 6, 3000, 64)
    case = G.make_case(1, 2, 512, 64, False, seed=45)
    want = G.bwd(case, "shift")
    dash.dash_set_spin_limit_us(2000)
    dash.dash_inject_fault(1)
    dash.dash_inject_fault(2)
    dash.dash_attn_bwd(*[case[n] for n in ("q", "k", "v", "o", "do", "lse")], False, "shift")
    dash.dash_attn_sparse_fwd(q, k, v, idx, 64, plan=plan)
    assert [dash.dash_attn_sync_status() for _ in range(3)] == [TIMEOUT, TIMEOUT, 0]
    dash.dash_set_spin_limit_us(0)
    for a, b in zip(G.bwd(case, "shift"), want):
        assert torch.equal(a, b)
