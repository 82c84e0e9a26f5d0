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
