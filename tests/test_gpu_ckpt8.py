"""8-bit checkpoints on the GPU: the stored bytes and the values read back equal the 64-bit form, and
the backward from checkpoints is bitwise the backward on the values they stand for."""
import pytest
import torch

from persistent_sm_attn_b200 import binding as dash
from tests import sparse_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def check(x):
    (m, e), = dash.dash_ckpt8_pack(x)
    wm, we = R.ckpt_pack(x)
    assert torch.equal(e, we) and torch.equal(m, wm)
    back, = dash.dash_ckpt8_unpack((m, e))
    assert back.dtype == torch.bfloat16
    assert torch.equal(back.double().nan_to_num(123.0), R.ckpt_values(m, e).nan_to_num(123.0))
    return back


@pytest.mark.parametrize("shape", [(32,), (1, 32), (3, 64), (2, 3, 77, 128), (5, 1, 1, 96), (300, 4096)])
def test_round_trip(shape):
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    back = check(x)
    # half a step of 2^e, a whole one where 127 clamps; 2^e <= max|x| 2^-6
    top = x.double().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True)
    assert ((back.double() - x.double()).unflatten(-1, (-1, 32)).abs() <= top * 2.0 ** -6).all()


def test_every_bf16_value_as_a_group_maximum():
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    g = torch.zeros(65536, 32, device="cuda", dtype=torch.bfloat16)
    g[:, 7] = x
    g[:, 8] = (x.float() * 0.3).to(torch.bfloat16)
    g[:, 9] = -g[:, 8]
    back = check(g)
    bad = ~torch.isfinite(x.float())
    assert torch.isnan(back[bad].float()).all() and torch.isfinite(back[~bad].float()).all()


def test_empty_and_several_tensors():
    gen = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
          for s in ((2, 64), (0, 32), (7, 32), (1, 5, 128), (3, 96), (4, 32))]
    pairs = dash.dash_ckpt8_pack(*xs)
    back = dash.dash_ckpt8_unpack(*pairs)
    for x, (m, e), y in zip(xs, pairs, back):
        assert m.shape == x.shape and y.shape == x.shape
        if x.numel():
            assert torch.equal(m, R.ckpt_pack(x)[0]) and torch.equal(e, R.ckpt_pack(x)[1])
            assert torch.equal(y.double(), R.ckpt_values(m, e))
    assert dash.dash_ckpt8_pack() == [] and dash.dash_ckpt8_unpack() == []


def test_halves_and_clamps():
    # groups with a maximum of 64 to 127.5 steps beside every half step below it, either sign
    top = torch.arange(128, 256, device="cuda") / 2
    half = torch.arange(128, device="cuda").view(1, -1) + 0.5
    vals = torch.minimum(half.expand(128, 128), top.view(-1, 1))
    g = torch.stack([top.view(-1, 1).expand(128, 128), vals, -vals, -top.view(-1, 1).expand(128, 128)], -1)
    x = torch.zeros(128 * 128, 32, device="cuda")
    x[:, [0, 13, 22, 31]] = g.reshape(-1, 4).float()
    for e in (-126, -20, 0, 60):
        check((x * 2.0 ** e).to(torch.bfloat16))


def test_tensors_that_end_inside_a_chunk():
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn(s, 32, generator=gen, device="cuda").to(torch.bfloat16)
          for s in (129, 5, 515, 32, 64, 1, 31)]
    for x, (m, e), y in zip(xs, pairs := dash.dash_ckpt8_pack(*xs), dash.dash_ckpt8_unpack(*pairs)):
        assert torch.equal(m, R.ckpt_pack(x)[0]) and torch.equal(e, R.ckpt_pack(x)[1])
        assert torch.equal(y.double(), R.ckpt_values(m, e))


@pytest.mark.parametrize("H,Hkv,S,D,causal,schedule", [
    (2, 2, 256, 64, True, "sym_shift"), (2, 2, 256, 128, False, "shift"), (4, 1, 384, 64, False, "shift"),
    (2, 2, 256, 64, False, "shift_pairs")])
def test_backward_from_checkpoints(H, Hkv, S, D, causal, schedule):
    gen = torch.Generator(device="cuda").manual_seed(5)
    mk = lambda h: torch.randn(2, h, S, D, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v, do = mk(H), mk(Hkv), mk(Hkv), mk(H)
    o, lse = dash.dash_attn_fwd_gqa(q, k, v, causal)
    packed = dash.dash_ckpt8_pack(q, k, v, o)
    got = dash.dash_attn_bwd_ckpt8(*packed, do, lse, causal, schedule)
    vals = [R.ckpt_values(m, e).to(torch.bfloat16) for m, e in packed]
    fn = dash.dash_attn_bwd if H == Hkv else dash.dash_attn_bwd_gqa
    want = fn(*vals, do, lse, causal, schedule)
    assert dash.dash_attn_sync_status() == 0
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_the_backward_takes_checkpoints_of_four_dimensions():
    x = torch.zeros(64, device="cuda", dtype=torch.bfloat16)
    packed = dash.dash_ckpt8_pack(x, x, x, x)
    with pytest.raises(ValueError, match="q must be"):
        dash.dash_attn_bwd_ckpt8(*packed, x, torch.zeros(1, device="cuda"), True)


def test_the_error_is_half_a_step():
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(5000, 256, generator=gen, device="cuda").to(torch.bfloat16)
    back = check(x)
    # elements up to 127.5 steps; a bf16 in [64, 128) steps is a whole number of halves, so the clamp
    # to 127 costs half a step as well.  A step is at most max|x| 2^-6
    g = x.double().unflatten(-1, (-1, 32))
    off = (back.double() - x.double()).unflatten(-1, (-1, 32)).abs()
    assert (off <= g.abs().amax(-1, keepdim=True) * 2.0 ** -7).all()
