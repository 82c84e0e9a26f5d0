"""Refusals of the sparse calls and of the checkpoints, without a GPU: by the binding before anything
reaches the library, and by the library before anything reaches the device."""
import ctypes

import pytest
import torch

from persistent_sm_attn_b200 import binding as dash

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def al():
    buf = ctypes.create_string_buffer(64)
    test_buffers.append(buf)
    return (ctypes.addressof(buf) + 15) // 16 * 16


test_buffers = []
SHAPE = dict(B=1, H=4, Hkv=2, Sq=8, Sk=256, D=64, block=64, topk=2, causal=1)


def fwd(lib, al, ptr=None, strides=None, scale=0.0, plan=None, work=None, **kw):
    s = dict(SHAPE, **kw)
    p = al if ptr is None else ptr
    return lib.dash_attn_sparse_fwd(p, al, al, strides, al if plan is None else plan, al, al,
                                    al if work is None else work, s["B"], s["H"], s["Hkv"], s["Sq"],
                                    s["Sk"], s["D"], s["block"], s["topk"], s["causal"], scale, None)


def tokens(lib, al, ptr=None, strides=None, scale=0.0, idx=None, **kw):
    s = dict(SHAPE, **kw)
    return lib.dash_attn_sparse_tokens(al if ptr is None else ptr, al, al, strides,
                                       al if idx is None else idx, None, None, al, al, s["B"], s["H"],
                                       s["Hkv"], s["Sq"], s["Sk"], s["D"], s["block"], s["topk"],
                                       s["causal"], scale, None)


def bwd(lib, al, ptr=None, strides=None, scale=0.0, **kw):
    s = dict(SHAPE, **kw)
    return lib.dash_attn_sparse_bwd(al if ptr is None else ptr, al, al, al, strides, al, al, al, al, al,
                                    al, al, s["B"], s["H"], s["Hkv"], s["Sq"], s["Sk"], s["D"],
                                    s["block"], s["topk"], s["causal"], scale, None)


@pytest.mark.parametrize("call", [fwd, tokens, bwd])
def test_attention_refuses(lib, al, call):
    assert call(lib, al, ptr=0) == INVALID
    assert call(lib, al, ptr=al + 2) == INVALID            # misaligned
    assert call(lib, al, D=96) == UNSUPPORTED
    assert call(lib, al, Hkv=3) == INVALID                 # heads do not divide
    assert call(lib, al, Hkv=0) == INVALID
    assert call(lib, al, H=258, Hkv=2) == UNSUPPORTED      # more than 128 heads of a K/V head
    for bad in (dict(B=-1), dict(Sq=-1), dict(Sk=0), dict(topk=0), dict(block=0), dict(block=96),
                dict(block=-64), dict(causal=2), dict(causal=-1)):
        assert call(lib, al, **bad) == INVALID, bad
    for scale in (-1.0, float("nan"), float("inf")):
        assert call(lib, al, scale=scale) == INVALID
    n = 12 if call is bwd else 9
    for bad in (0, 4, -8, 12, 1 << 38):
        flat = [512, 64, 64] * (n // 3)
        flat[1] = bad                                      # the stride of q's heads
        assert call(lib, al, strides=(ctypes.c_longlong * n)(*flat)) == INVALID, bad
    assert call(lib, al, B=1 << 20, H=1 << 10, Hkv=1 << 10, Sq=1 << 10) == UNSUPPORTED
    # nothing to do: the pointers are not looked at
    assert call(lib, 0, B=0) == OK
    assert call(lib, 0, H=0) == OK
    if call is not bwd:
        assert call(lib, 0, Sq=0) == OK


def test_limits_of_the_call_without_a_plan(lib, al):
    assert tokens(lib, al, topk=1025) == UNSUPPORTED
    assert tokens(lib, al, Sk=65537 * 64) == UNSUPPORTED
    assert tokens(lib, al, idx=0) == INVALID


def test_plan_refuses(lib, al):
    s = (1, 4, 2, 8, 256, 64, 2)
    assert lib.dash_sparse_plan_bytes(*s) > 0
    assert lib.dash_sparse_plan(al, None, None, 0, *s, 1, None) == INVALID
    assert lib.dash_sparse_plan(0, None, None, al, *s, 1, None) == INVALID
    assert lib.dash_sparse_plan(al, al + 2, None, al, *s, 1, None) == INVALID
    assert lib.dash_sparse_plan(al, None, None, al, *s, 2, None) == INVALID
    assert lib.dash_sparse_plan_bytes(1, 4, 2, 8, 256, 100, 2) == -INVALID
    # one tile's masks have to fit in shared memory
    assert lib.dash_sparse_plan_bytes(1, 1, 1, 256, 1 << 23, 64, 2) == -UNSUPPORTED
    assert lib.dash_attn_sparse_work_bytes(1, 4, 2, 8, 256, 96, 64, 2, 0) == -UNSUPPORTED
    assert lib.dash_attn_sparse_work_bytes(0, 4, 2, 8, 256, 64, 64, 2, 1) == 0


def test_selection_refuses(lib, al):
    def means(k=al, B=1, Hkv=2, Sk=256, D=64, block=64, out=al, n=None):
        return lib.dash_block_means(k, None, out, n, None, B, Hkv, Sk, D, block, None)

    assert means(k=0) == INVALID and means(k=al + 8) == INVALID and means(out=al + 2) == INVALID
    assert means(n=al + 1) == INVALID
    assert means(block=32) == INVALID and means(block=65) == INVALID and means(Sk=0) == INVALID
    assert means(D=32) == UNSUPPORTED and means(B=70000) == UNSUPPORTED
    assert means(k=0, B=0) == OK

    def select(q=al, B=1, H=4, Hkv=2, Sq=8, Sk=256, D=64, block=64, topk=4, causal=1, sink=1, local=1):
        return lib.dash_block_select(q, None, al, al, None, None, B, H, Hkv, Sq, Sk, D, block, topk,
                                     causal, sink, local, None)

    assert select(q=0) == INVALID and select(causal=3) == INVALID and select(topk=0) == INVALID
    assert select(sink=3, local=2) == INVALID                  # more than topk
    assert select(sink=-1) == INVALID and select(local=-1) == INVALID
    assert select(sink=2 ** 31 - 1, local=2 ** 31 - 1) == INVALID
    assert select(Sk=4097 * 64) == UNSUPPORTED and select(D=256) == UNSUPPORTED
    assert select(q=0, Sq=0) == OK


def test_sizes_that_pass_32_bits(lib, al):
    for call in (fwd, tokens, bwd):
        assert call(lib, al, Sk=(1 << 30) + 64, block=1 << 30) == UNSUPPORTED
        assert call(lib, al, block=2 ** 31 - 64) == UNSUPPORTED
        assert call(lib, al, topk=(1 << 20) + 1) == UNSUPPORTED
    assert lib.dash_sparse_plan_bytes(1, 4, 2, 8, 256, 2 ** 31 - 64, 2) == -UNSUPPORTED
    assert lib.dash_block_means(al, None, al, None, None, 1, 2, 256, 64, 2 ** 31 - 64, None) == UNSUPPORTED
    assert lib.dash_block_select(al, None, al, al, None, None, 1, 4, 2, 8, 256, 64, 2 ** 31 - 64, 4, 1, 1,
                                 1, None) == UNSUPPORTED
    # a Python integer past the entry points' int does not arrive as another one
    q, k = host(1, 4, 8, 64), host(1, 2, 256, 64)
    means, idx = host(1, 2, 1, 64, dtype=torch.float32), host(1, 2, 8, 2, dtype=torch.int32)
    for block in (2 ** 31, 2 ** 32 + 64):
        with pytest.raises(ValueError):
            dash._block_count(256, block)
    with pytest.raises(ValueError):
        dash._block_count(2 ** 32 + 256, 64)
    for bad in (dict(topk=2 ** 32 + 1), dict(sink=2 ** 32), dict(local=2 ** 32 + 1), dict(topk=0)):
        with pytest.raises(ValueError, match="topk"):
            dash.dash_block_select(q, means, 256, 256, **dict(dict(topk=2), **bad))
    with pytest.raises(ValueError):
        dash.dash_sparse_plan(idx, 2 ** 32 + 4, 256, 64)


def test_checkpoints_refuse(lib, al):
    vp, ll = ctypes.c_void_p * 1, ctypes.c_longlong * 1
    for call in (lib.dash_ckpt8_pack, lib.dash_ckpt8_unpack):
        mid = (vp(al), vp(al)) if call is lib.dash_ckpt8_pack else (vp(al), vp(al))
        assert call(vp(al), *mid, ll(33), 1, None) == INVALID   # not whole groups
        assert call(vp(al), *mid, ll(-32), 1, None) == INVALID
        assert call(vp(0), *mid, ll(32), 1, None) == INVALID
        assert call(vp(al), *mid, ll(32), 0, None) == INVALID
        assert call(vp(al), *mid, ll(32), 5, None) == INVALID
        assert call(None, *mid, ll(32), 1, None) == INVALID
        assert call(vp(0), vp(0), vp(0), ll(0), 1, None) == OK


def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_the_binding_takes_device_tensors_only():
    q, k = host(1, 4, 8, 64), host(1, 2, 256, 64)
    idx = host(1, 2, 8, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dash.dash_attn_sparse_fwd(q, k, k, idx, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dash.dash_sparse_plan(idx, 4, 256, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dash.dash_block_means(k, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dash.dash_block_select(q, host(1, 2, 4, 64, dtype=torch.float32), 256, 64, 2)
    with pytest.raises(ValueError, match="CUDA"):
        dash.dash_ckpt8_pack(q)
    with pytest.raises(ValueError, match="CUDA"):
        dash.dash_ckpt8_unpack((host(1, 64, dtype=torch.int8), host(1, 2, dtype=torch.int8)))


@pytest.mark.parametrize("bad", [
    dict(shape=(1, 4, 8, 128)), dict(dtype=torch.float16)])
def test_the_binding_looks_at_shapes_and_types_first(bad):
    with pytest.raises(ValueError, match="has (shape|dtype)"):
        dash._expect("x", host(*bad.get("shape", (1, 4, 8, 64)), dtype=bad.get("dtype", torch.bfloat16)),
                     (1, 4, 8, 64), torch.bfloat16)


def test_names_are_public():
    import persistent_sm_attn_b200 as pkg
    for name in ("dash_block_means", "dash_block_select", "dash_sparse_plan", "dash_attn_sparse_fwd",
                 "dash_attn_sparse_bwd", "dash_attn_sparse_bwd_ckpt8", "dash_ckpt8_pack",
                 "dash_ckpt8_unpack", "dash_attn_bwd_ckpt8"):
        assert getattr(pkg, name) is getattr(dash, name)


def test_a_plan_of_another_selection_is_refused():
    idx = host(1, 2, 8, 3, dtype=torch.int32)
    n = host(1, dtype=torch.int32)
    plan = dash.SparsePlan(None, (1, 4, 2, 8, 256, 64, 3), True, 0, True, False)
    same = dash._expect_same_selection
    same(plan, idx, 64, True, n, None)
    same(plan, None, 64, None, None, None)
    for bad, what in (((plan, idx, 128, True, n, None), "blocks of 64"),
                      ((plan, idx, 64, False, n, None), "causal"),
                      ((plan, idx[..., :2], 64, True, n, None), "idx"),
                      ((plan, idx, 64, True, n, n), "q_start"),
                      ((dash.SparsePlan(None, plan.shape, True, 0, False, True), idx, 64, True, n, n), "kv_len")):
        with pytest.raises(ValueError, match=what):
            same(*bad)


@pytest.mark.parametrize("call", [fwd, tokens])
def test_no_queries_before_strided_keys(lib, al, call):
    # one sequence without queries: q's contiguous strides are 0, which is no one's fault
    flat = (ctypes.c_longlong * 9)(*([64, 64, 64] + [65536, 72, 144] * 2))
    assert call(lib, al, strides=flat, Sq=0) == OK
    flat[7] = 12                                           # v's heads: still looked at
    assert call(lib, al, strides=flat, Sq=0) == INVALID


def test_a_selection_needs_a_query_head(lib, al):
    call = lambda B=1, H=0, Hkv=2, Sq=8: lib.dash_block_select(
        al, None, al, al, None, None, B, H, Hkv, Sq, 256, 64, 64, 4, 1, 1, 1, None)
    assert call() == INVALID                       # places in idx that nothing would fill
    assert call(B=0) == OK and call(Sq=0) == OK and call(Hkv=0) == OK


def test_a_scale_of_zero_is_not_the_default():
    assert dash._scale(None) == 0.0 and dash._scale(0.25) == 0.25 and dash._scale(2) == 2.0
    for scale in (0, 0.0, -0.0, 1e-50):  # the last is 0 in fp32
        with pytest.raises(ValueError, match="scale"):
            dash._scale(scale)
    # negative, infinite and NaN scales are refused by the C calls
