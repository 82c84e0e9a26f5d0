"""ctypes binding of libdash_attn.so (argument marshalling only).

Every step of the backward runs in the library's CUDA kernels; this module
turns torch tensors into pointers and a stream handle, and raises
``DashError`` on a non-zero status.  It never falls back to another
implementation: if the library is missing or fails to load, ``load()``
raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdash_attn.so")

SCHEDULES = {"naive_asc": 0, "descending": 1, "shift": 2, "sym_shift": 3, "atomic": 4,
             "shift_pairs": 5, "sym_shift_pairs": 6}
STATUS = {0: "DASH_OK", 1: "DASH_ERR_INVALID_ARG", 2: "DASH_ERR_UNSUPPORTED", 3: "DASH_ERR_CUDA",
          4: "DASH_ERR_TIMEOUT", 5: "DASH_ERR_OOM", 6: "DASH_ERR_SCHEDULE"}

EXPORTS = ("dash_attn_fwd", "dash_attn_bwd", "dash_attn_sync_status", "dash_status_string",
           "dash_set_spin_limit_us", "dash_bwd_num_ctas", "dash_release_workspace",
           "dash_sched_table", "dash_sched_simulate", "dash_sched_simulate_gqa",
           "dash_dag_longest_path",
           "dash_profile_begin", "dash_profile_end", "dash_attn_bwd_noalloc",
           "dash_trace_bwd", "dash_inject_fault", "dash_sched_check", "dash_attn_bwd_host",
           "dash_sched_table_part", "dash_attn_fwd_gqa", "dash_attn_bwd_gqa",
           "dash_sched_table_gqa", "dash_attn_noalloc_sync_status",
           "dash_attn_bwd_gqa_split", "dash_bwd_gqa_split_for", "dash_set_dq_chain_mode",
           "dash_dq_chain_uses_red", "dash_set_head_interleave",
           "dash_bwd_head_interleave", "dash_set_slot_placement",
           "dash_slot_placement_by_smid", "dash_sched_table_pairs",
           "dash_block_means", "dash_block_select", "dash_sparse_plan_bytes",
           "dash_sparse_plan", "dash_attn_sparse_work_bytes", "dash_attn_sparse_fwd",
           "dash_attn_sparse_bwd", "dash_attn_sparse_tokens", "dash_ckpt8_pack",
           "dash_ckpt8_unpack")


class DashError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


_lib = None


def load(path: str | None = None):
    """Load (building first if absent or stale) the shared library."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    if path is None:
        from . import build as _build
        try:
            _build.build()
        except Exception as e:  # no compiler on this machine: use what is there
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libdash_attn.so is missing and could not be built: {e}")
        path = LIB_PATH
    lib = ctypes.CDLL(path)
    vp, i, ll, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_double
    P = ctypes.POINTER
    lib.dash_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.dash_attn_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, i, vp]
    lib.dash_attn_bwd_noalloc.argtypes = [vp] * 9 + [i, i, i, i, i, i, vp]
    lib.dash_attn_bwd_host.argtypes = [vp] * 9 + [i, i, i, i, i, i, vp]
    lib.dash_attn_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.dash_attn_bwd_gqa.argtypes = [vp] * 9 + [i, i, i, i, i, i, i, vp]
    lib.dash_attn_bwd_gqa_split.argtypes = [vp] * 9 + [i, i, i, i, i, i, i, i, vp]
    lib.dash_bwd_gqa_split_for.argtypes = [i, i, i, i, i, i, i, P(i)]
    lib.dash_set_dq_chain_mode.argtypes = [i]
    lib.dash_dq_chain_uses_red.argtypes = [i, i, i, i, P(i)]
    lib.dash_set_head_interleave.argtypes = [i]
    lib.dash_set_slot_placement.argtypes = [i]
    lib.dash_slot_placement_by_smid.argtypes = [i, P(i)]
    lib.dash_bwd_head_interleave.argtypes = [i, i, i, i, i, i, P(i)]
    lib.dash_attn_sync_status.argtypes = [vp]
    lib.dash_attn_noalloc_sync_status.argtypes = [vp]
    lib.dash_status_string.argtypes = [i]
    lib.dash_status_string.restype = ctypes.c_char_p
    lib.dash_set_spin_limit_us.argtypes = [ll]
    lib.dash_inject_fault.argtypes = [i]
    lib.dash_bwd_num_ctas.argtypes = [i, i, P(i)]
    lib.dash_release_workspace.argtypes = []
    lib.dash_sched_table.argtypes = [i, i, i, i, i, vp, ll]
    lib.dash_sched_table.restype = ll
    lib.dash_sched_table_part.argtypes = [i, i, i, i, i, i, i, vp, ll]
    lib.dash_sched_table_part.restype = ll
    lib.dash_sched_table_gqa.argtypes = [i, i, i, i, i, i, vp, ll]
    lib.dash_sched_table_gqa.restype = ll
    lib.dash_sched_table_pairs.argtypes = [i, i, i, i, vp, ll]
    lib.dash_sched_table_pairs.restype = ll
    lib.dash_sched_simulate.argtypes = [i, i, i, i, i, d, d, i, i, P(d), P(d), P(d), P(ll)]
    lib.dash_sched_simulate_gqa.argtypes = [i, i, i, i, i, i, d, d, i, i, P(d), P(d), P(d),
                                            P(ll)]
    lib.dash_sched_check.argtypes = [i, i, i, i, vp, ll]
    lib.dash_dag_longest_path.argtypes = [i, i, vp, vp, vp, vp, vp, P(d)]
    lib.dash_trace_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, i, vp, vp, ll, P(i), P(i)]
    f = ctypes.c_float
    lib.dash_block_means.argtypes = [vp] * 5 + [i] * 5 + [vp]
    lib.dash_block_select.argtypes = [vp] * 6 + [i] * 11 + [vp]
    lib.dash_sparse_plan_bytes.argtypes = [i] * 7
    lib.dash_sparse_plan.argtypes = [vp] * 4 + [i] * 8 + [vp]
    lib.dash_attn_sparse_work_bytes.argtypes = [i] * 9
    lib.dash_attn_sparse_fwd.argtypes = [vp] * 8 + [i] * 9 + [f, vp]
    lib.dash_attn_sparse_tokens.argtypes = [vp] * 9 + [i] * 9 + [f, vp]
    lib.dash_attn_sparse_bwd.argtypes = [vp] * 12 + [i] * 9 + [f, vp]
    lib.dash_ckpt8_pack.argtypes = [vp, vp, vp, vp, i, vp]
    lib.dash_ckpt8_unpack.argtypes = [vp, vp, vp, vp, i, vp]
    for name in ("dash_sparse_plan_bytes", "dash_attn_sparse_work_bytes"):
        getattr(lib, name).restype = ll
    lib.dash_profile_begin.argtypes = []
    lib.dash_profile_end.argtypes = [P(d), P(d), P(ll)]
    for name in EXPORTS:
        if name not in ("dash_status_string", "dash_sched_table", "dash_sched_table_part",
                        "dash_sched_table_gqa", "dash_attn_noalloc_sync_status",
                        "dash_sched_table_pairs", "dash_sparse_plan_bytes",
                        "dash_attn_sparse_work_bytes"):
            getattr(lib, name).restype = ctypes.c_int
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != 0:
        raise DashError(rc, what)


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _sched_id(schedule) -> int:
    return SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)


def _check_tensors(q, k, v, o=None, do=None, lse=None, outs=(), *, cuda=True, gqa=False):
    """Reject tensors whose shape, dtype, layout or device differs from what the C
    entry points read and write: q [B,H,S,D] bf16; k, v [B,Hkv,S,D] bf16 (Hkv = H
    unless gqa); o, do like q; lse [B,H,S] fp32; outs (dq, dk, dv) or (o, lse).
    The C ABI takes bare pointers, so a mismatch here would otherwise become an
    out-of-bounds device access."""
    import torch
    if q.dim() != 4:
        raise ValueError("q must be [B,H,S,D]")
    B, H, S, D = q.shape
    Hkv = k.shape[1] if gqa and k.dim() == 4 else H
    bf, f32 = torch.bfloat16, torch.float32
    want = [("q", q, (B, H, S, D), bf), ("k", k, (B, Hkv, S, D), bf), ("v", v, (B, Hkv, S, D), bf)]
    if o is not None:
        want.append(("o", o, (B, H, S, D), bf))
    if do is not None:
        want.append(("do", do, (B, H, S, D), bf))
    if lse is not None:
        want.append(("lse", lse, (B, H, S), f32))
    names = ("dq", "dk", "dv") if len(outs) == 3 else ("out", "lse_out")
    shapes = ((B, H, S, D), (B, Hkv, S, D), (B, Hkv, S, D)) if len(outs) == 3 else \
        ((B, H, S, D), (B, H, S))
    dtypes = (bf, bf, bf) if len(outs) == 3 else (bf, f32)
    want += [(n, t, sh, dt) for n, t, sh, dt in zip(names, outs, shapes, dtypes) if t is not None]
    for name, t, shape, dtype in want:
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if cuda and (not t.is_cuda or t.device != q.device):
            raise ValueError(f"{name} must be a CUDA tensor on {q.device}")
        if not cuda and t.is_cuda:
            raise ValueError(f"{name} must be a host tensor")


def dash_status_string(status: int) -> str:
    return load().dash_status_string(int(status)).decode()


def dash_attn_fwd(q, k, v, causal: bool, out=None, lse=None, stream=None):
    """O, LSE = attention forward (bf16 [B,H,S,D] CUDA tensors)."""
    import torch
    _check_tensors(q, k, v, outs=(out, lse))
    B, H, S, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    rc = load().dash_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                              int(bool(causal)), _stream_handle(stream))
    _check(rc, "dash_attn_fwd")
    return out, lse


def dash_attn_bwd(q, k, v, o, do, lse, causal: bool, schedule="shift", dq=None, dk=None,
                  dv=None, stream=None):
    """dQ, dK, dV of attention (bf16 [B,H,S,D], lse fp32 [B,H,S]; CUDA tensors)."""
    import torch
    _check_tensors(q, k, v, o, do, lse, (dq, dk, dv))
    B, H, S, D = q.shape
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    rc = load().dash_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, H, S, D, int(bool(causal)),
                              _sched_id(schedule), _stream_handle(stream))
    _check(rc, "dash_attn_bwd")
    return dq, dk, dv


def dash_attn_fwd_gqa(q, k, v, causal: bool, out=None, lse=None, stream=None):
    """O, LSE of grouped-query attention: q [B,H,S,D], k and v [B,Hkv,S,D] (bf16
    CUDA tensors), query head h reading K/V head h // (H // Hkv)."""
    import torch
    _check_tensors(q, k, v, outs=(out, lse), gqa=True)
    B, H, S, D = q.shape
    Hkv = k.shape[1]
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    rc = load().dash_attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, S,
                                  D, int(bool(causal)), _stream_handle(stream))
    _check(rc, "dash_attn_fwd_gqa")
    return out, lse


def dash_attn_bwd_gqa(q, k, v, o, do, lse, causal: bool, schedule="shift", dq=None, dk=None,
                      dv=None, stream=None, split=None):
    """dQ [B,H,S,D], dK and dV [B,Hkv,S,D] of grouped-query attention (dK, dV summed
    over each K/V head's query heads).  split: sub-groups per K/V head (a power of
    two dividing H / Hkv); None or 0 lets the library choose."""
    import torch
    _check_tensors(q, k, v, o, do, lse, (dq, dk, dv), gqa=True)
    B, H, S, D = q.shape
    Hkv = k.shape[1]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
            _ptr(dv), B, H, Hkv, S, D, int(bool(causal)), _sched_id(schedule))
    if split is None:
        rc = load().dash_attn_bwd_gqa(*args, _stream_handle(stream))
    else:
        rc = load().dash_attn_bwd_gqa_split(*args, int(split), _stream_handle(stream))
    _check(rc, "dash_attn_bwd_gqa")
    return dq, dk, dv


def dash_bwd_gqa_split_for(num_ctas: int, B: int, Hkv: int, group: int, S: int, causal: bool,
                           schedule="shift") -> int:
    """The sub-group count dash_attn_bwd_gqa chooses (host only)."""
    n = ctypes.c_int(0)
    _check(load().dash_bwd_gqa_split_for(num_ctas, B, Hkv, group, S, int(bool(causal)),
                                         _sched_id(schedule), ctypes.byref(n)),
           "dash_bwd_gqa_split_for")
    return n.value


def dash_attn_bwd_host(q, k, v, o, do, lse, causal: bool, schedule="shift", dq=None, dk=None,
                       dv=None, stream=None):
    """The backward from host (CPU) tensors, pipelined over parts of the heads;
    results are bitwise those of dash_attn_bwd.  Page-locked tensors let the
    copies overlap the compute.  The outputs are valid once `stream` (default:
    torch's current stream) has completed."""
    import torch
    _check_tensors(q, k, v, o, do, lse, (dq, dk, dv), cuda=False)
    B, H, S, D = q.shape
    pin = q.is_pinned()
    dq = torch.empty(q.shape, dtype=q.dtype, pin_memory=pin) if dq is None else dq
    dk = torch.empty(k.shape, dtype=k.dtype, pin_memory=pin) if dk is None else dk
    dv = torch.empty(v.shape, dtype=v.dtype, pin_memory=pin) if dv is None else dv
    rc = load().dash_attn_bwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv), B, H, S, D, int(bool(causal)),
                                   _sched_id(schedule), _stream_handle(stream))
    _check(rc, "dash_attn_bwd_host")
    return dq, dk, dv


def dash_attn_bwd_noalloc(q, k, v, o, do, lse, causal: bool, schedule, dq, dk, dv,
                          stream=None):
    """The backward through the entry point that allocates no device memory.
    Outputs must be preallocated; all scratch comes from the library's static
    device array (see include/dash_attn.h)."""
    for t in (dq, dk, dv):
        if t is None:
            raise ValueError("dash_attn_bwd_noalloc needs preallocated dq, dk, dv")
    _check_tensors(q, k, v, o, do, lse, (dq, dk, dv))
    B, H, S, D = q.shape
    rc = load().dash_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                      _ptr(dq), _ptr(dk), _ptr(dv), B, H, S, D,
                                      int(bool(causal)), _sched_id(schedule),
                                      _stream_handle(stream))
    _check(rc, "dash_attn_bwd_noalloc")
    return dq, dk, dv


def dash_attn_sync_status(stream=None) -> int:
    return int(load().dash_attn_sync_status(_stream_handle(stream)))


def dash_attn_noalloc_sync_status(stream=None) -> int:
    """Waits for the stream and returns (and clears) the status that
    dash_attn_bwd_noalloc's calls recorded on the current device."""
    return int(load().dash_attn_noalloc_sync_status(_stream_handle(stream)))


def dash_set_spin_limit_us(us: int) -> None:
    _check(load().dash_set_spin_limit_us(int(us)), "dash_set_spin_limit_us")


def dash_inject_fault(mode: int) -> None:
    """Arm the host-side fault for the next backward (1) or block-sparse call with a plan (2), or
    cancel both (0)."""
    _check(load().dash_inject_fault(int(mode)), "dash_inject_fault")


def dash_bwd_num_ctas(device: int = 0, D: int = 128) -> int:
    n = ctypes.c_int(0)
    _check(load().dash_bwd_num_ctas(device, D, ctypes.byref(n)), "dash_bwd_num_ctas")
    return n.value


def dash_set_dq_chain_mode(mode: int) -> None:
    """0: the library picks per launch; 1: middle positions of the ordered dQ chains
    add with red in L2; 2: load-add-store on the SM (bitwise the same results)."""
    _check(load().dash_set_dq_chain_mode(int(mode)), "dash_set_dq_chain_mode")


def dash_dq_chain_uses_red(schedule: str, S: int, D: int = 128, heads_per_unit: int = 1) -> bool:
    """Whether a deterministic backward of this schedule, length and head dim, with this
    many query heads per unit of its table, adds its chains' middle positions with red
    under the current mode (host only)."""
    r = ctypes.c_int(0)
    _check(load().dash_dq_chain_uses_red(_sched_id(schedule), S, int(D), int(heads_per_unit),
                                         ctypes.byref(r)),
           "dash_dq_chain_uses_red")
    return bool(r.value)


def dash_set_slot_placement(mode: int) -> None:
    """1: each CTA runs the table slot of its SM id's rank; 2: CTA b runs slot b; 0:
    the library's choice (by SM id from 128 tiles).  Bitwise the same results."""
    _check(load().dash_set_slot_placement(int(mode)), "dash_set_slot_placement")


def dash_slot_placement_by_smid(S: int) -> bool:
    """Whether a backward of length S places the table's slots by SM id under the
    current mode (host only)."""
    r = ctypes.c_int(0)
    _check(load().dash_slot_placement_by_smid(int(S), ctypes.byref(r)),
           "dash_slot_placement_by_smid")
    return bool(r.value)


def dash_set_head_interleave(mode: int) -> None:
    """Heads per unit of a multi-head backward's table: 0 the library's choice, 1 never
    interleave, 2 or 4 that many whenever it divides B * H."""
    _check(load().dash_set_head_interleave(int(mode)), "dash_set_head_interleave")


def dash_bwd_head_interleave(num_ctas: int, D: int, schedule: str, n_heads: int, S: int,
                             causal: bool) -> int:
    """Heads per unit a multi-head backward takes under the current mode (host only)."""
    r = ctypes.c_int(0)
    _check(load().dash_bwd_head_interleave(num_ctas, D, _sched_id(schedule), n_heads, S,
                                           int(bool(causal)), ctypes.byref(r)),
           "dash_bwd_head_interleave")
    return r.value


def dash_release_workspace() -> None:
    _check(load().dash_release_workspace(), "dash_release_workspace")


def dash_sched_table(n_heads: int, N: int, causal: bool, schedule, num_ctas: int):
    """Rows (cta, head, kv, q, position, chain_index) as a list of tuples."""
    lib = load()
    sid = _sched_id(schedule)
    n = lib.dash_sched_table(n_heads, N, int(bool(causal)), sid, num_ctas, None, 0)
    if n < 0:
        raise DashError(int(-n), "dash_sched_table")
    buf = (ctypes.c_int * (6 * n))()
    lib.dash_sched_table(n_heads, N, int(bool(causal)), sid, num_ctas, buf, n)
    flat = list(buf)
    return [tuple(flat[6 * r: 6 * r + 6]) for r in range(n)]


def dash_sched_table_part(n_heads: int, N: int, causal: bool, schedule, num_ctas: int,
                          h0: int, h1: int):
    """Rows of the part of the table covering heads [h0, h1), heads renumbered
    from 0, as the host-buffer path launches it."""
    lib = load()
    sid = _sched_id(schedule)
    n = lib.dash_sched_table_part(n_heads, N, int(bool(causal)), sid, num_ctas, h0, h1, None, 0)
    if n < 0:
        raise DashError(int(-n), "dash_sched_table_part")
    buf = (ctypes.c_int * (6 * max(n, 1)))()
    lib.dash_sched_table_part(n_heads, N, int(bool(causal)), sid, num_ctas, h0, h1, buf, n)
    flat = list(buf)
    return [tuple(flat[6 * r: 6 * r + 6]) for r in range(n)]


def dash_sched_table_gqa(n_heads: int, group: int, N: int, causal: bool, schedule,
                         num_ctas: int):
    """Rows (cta, query head, kv, q, position, chain_index) of a grouped-query table."""
    lib = load()
    sid = _sched_id(schedule)
    n = lib.dash_sched_table_gqa(n_heads, group, N, int(bool(causal)), sid, num_ctas, None, 0)
    if n < 0:
        raise DashError(int(-n), "dash_sched_table_gqa")
    buf = (ctypes.c_int * (6 * max(n, 1)))()
    lib.dash_sched_table_gqa(n_heads, group, N, int(bool(causal)), sid, num_ctas, buf, n)
    flat = list(buf)
    return [tuple(flat[6 * r: 6 * r + 6]) for r in range(n)]


def dash_sched_table_pairs(n_heads: int, N: int, causal: bool, num_ctas: int):
    """Rows (cta, head, kv, q, position, chain_index) of the grid's CTA-pair table
    (SHIFT_PAIRS, or SYM_SHIFT_PAIRS when causal) for num_ctas CTAs (even): CTAs 2i and
    2i + 1 run KV tiles 2m and 2m + 1 over the same Q tiles with the same positions."""
    lib = load()
    n = lib.dash_sched_table_pairs(n_heads, N, int(causal), num_ctas, None, 0)
    if n < 0:
        raise DashError(int(-n), "dash_sched_table_pairs")
    buf = (ctypes.c_int * (6 * max(n, 1)))()
    lib.dash_sched_table_pairs(n_heads, N, int(causal), num_ctas, buf, n)
    flat = list(buf)
    return [tuple(flat[6 * r: 6 * r + 6]) for r in range(n)]


def dash_sched_simulate(n_heads: int, N: int, causal: bool, schedule, num_ctas: int,
                        w_compute: float, w_reduce: float, dq_buffers: int = 0,
                        dq_chains: int = 1):
    """(critical_path, makespan, bubble_time, stalls) of a schedule's DAG;
    dq_chains = 2 models the kernel's two accumulators per dQ block."""
    cp, mk, bt = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    st = ctypes.c_longlong()
    rc = load().dash_sched_simulate(n_heads, N, int(bool(causal)), _sched_id(schedule), num_ctas,
                                    float(w_compute), float(w_reduce), int(dq_buffers),
                                    int(dq_chains), ctypes.byref(cp), ctypes.byref(mk),
                                    ctypes.byref(bt), ctypes.byref(st))
    _check(rc, "dash_sched_simulate")
    return cp.value, mk.value, bt.value, st.value


def dash_sched_simulate_gqa(n_heads: int, group: int, N: int, causal: bool, schedule,
                            num_ctas: int, w_compute: float, w_reduce: float,
                            dq_buffers: int = 0, dq_chains: int = 1):
    """dash_sched_simulate over the grouped-query table (`group` query heads per K/V head)."""
    cp, mk, bt = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    st = ctypes.c_longlong()
    rc = load().dash_sched_simulate_gqa(n_heads, group, N, int(bool(causal)), _sched_id(schedule),
                                        num_ctas, float(w_compute), float(w_reduce),
                                        int(dq_buffers), int(dq_chains), ctypes.byref(cp),
                                        ctypes.byref(mk), ctypes.byref(bt), ctypes.byref(st))
    _check(rc, "dash_sched_simulate_gqa")
    return cp.value, mk.value, bt.value, st.value


def dash_sched_check(n_heads: int, N: int, causal: bool, num_ctas: int, rows) -> int:
    """Status of the library's checks on a caller-supplied table given as rows
    (cta, head, kv, q, position, chain_index): 0 valid, 6 a failed check
    (coverage, positions or a deadlocking ticket order), 1 malformed rows."""
    flat = [int(x) for r in rows for x in r]
    buf = (ctypes.c_int * max(len(flat), 1))(*flat)
    return int(load().dash_sched_check(n_heads, N, int(bool(causal)), num_ctas, buf, len(rows)))


def dash_dag_longest_path(n_nodes: int, edges):
    """(cp, depth list, height list) of a weighted DAG given as (u, v, w) edges."""
    m = len(edges)
    src = (ctypes.c_int * max(m, 1))(*[e[0] for e in edges])
    dst = (ctypes.c_int * max(m, 1))(*[e[1] for e in edges])
    w = (ctypes.c_double * max(m, 1))(*[float(e[2]) for e in edges])
    depth = (ctypes.c_double * max(n_nodes, 1))()
    height = (ctypes.c_double * max(n_nodes, 1))()
    cp = ctypes.c_double()
    rc = load().dash_dag_longest_path(n_nodes, m, src, dst, w, depth, height, ctypes.byref(cp))
    _check(rc, "dash_dag_longest_path")
    return cp.value, list(depth)[:n_nodes], list(height)[:n_nodes]


def dash_profile_begin() -> None:
    _check(load().dash_profile_begin(), "dash_profile_begin")


def dash_profile_end():
    """(main kernel ms summed, auxiliary kernels ms summed, backward calls)."""
    m, a, n = ctypes.c_double(), ctypes.c_double(), ctypes.c_longlong()
    _check(load().dash_profile_end(ctypes.byref(m), ctypes.byref(a), ctypes.byref(n)),
           "dash_profile_end")
    return m.value, a.value, n.value


def dash_trace_bwd(q, k, v, o, do, lse, causal: bool, schedule="shift", stream=None):
    """One traced backward; returns (dq, dk, dv, trace [ctas, rows, 16] uint64 ns),
    the events per pair listed at dash_trace_bwd in include/dash_attn.h."""
    import numpy as np
    import torch
    _check_tensors(q, k, v, o, do, lse)
    B, H, S, D = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    N = S // 128
    EV = 16
    cap = EV * (B * H * N * N + 1024 * (N + 1))   # >= ctas * rows_per_cta * EV
    buf = np.zeros(cap, dtype=np.uint64)
    nc, rows = ctypes.c_int(), ctypes.c_int()
    rc = load().dash_trace_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                               _ptr(dk), _ptr(dv), B, H, S, D, int(bool(causal)),
                               _sched_id(schedule), _stream_handle(stream),
                               buf.ctypes.data_as(ctypes.c_void_p), cap, ctypes.byref(nc),
                               ctypes.byref(rows))
    _check(rc, "dash_trace_bwd")
    n = nc.value * rows.value * EV
    if n > cap:
        raise RuntimeError("trace buffer too small")
    return dq, dk, dv, buf[:n].reshape(nc.value, rows.value, EV)


# ---------------------------------------------------------------- block-sparse attention
# These calls run on the tensors' device, on `stream` or that device's current stream, and
# allocate what they return (and their scratch) on that stream.

class _Launch:
    """The device and stream of one call: tensors made inside belong to that stream."""
    __slots__ = ("_ctx", "_handle")

    def __init__(self, device, stream):
        import torch
        self._ctx = None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self._ctx, self._handle = torch.cuda.stream(stream), stream.cuda_stream
        else:
            if device.index != torch.cuda.current_device():
                self._ctx = torch.cuda.device(device)
            # the handle without the two objects of the public call (2 us); the name is torch's
            # own, so a torch may come without it
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            self._handle = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self._handle

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


def _expect(name, t, shape, dtype, device=None, contiguous=True):
    """Reject what the C entry point would misread: shape, dtype, device, layout."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on {device}" if device else ""))
    if contiguous:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return
    if t.data_ptr() % 16 and t.numel():
        raise ValueError(f"{name} must be 16-byte aligned")
    if t.is_contiguous():
        return
    shape, strides = t.shape, t.stride()
    if t.numel() and strides[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if t.numel() and any(n > 1 and (st < 8 or st % 8) for n, st in zip(shape[:-1], strides[:-1])):
        raise ValueError(f"{name} has strides {tuple(strides)}: positive multiples of 8 are "
                         "needed (no broadcast dimensions)")


def _expect_rows(name, t, B, device):
    """An optional int32 [B] tensor of the batch (kv_len, q_start, start)."""
    if t is None:
        return None
    import torch
    if not (t.dtype is torch.int32 and t.is_cuda and t.device == device and t.shape == (B,)
            and t.is_contiguous()):
        _expect(name, t, (B,), torch.int32, device)
    return t.data_ptr()


def _expect_input(name, t):
    """A bf16 input of any strides, of which only shape and device are its own; the strides
    argument.  The usual case at once (1 us in place of 3)."""
    import torch
    if t.dtype is torch.bfloat16 and t.is_cuda and t.is_contiguous() and not t.data_ptr() & 15:
        return None
    _expect(name, t, t.shape, torch.bfloat16, contiguous=False)
    return _strides(t)


def _like(t, dtype=None):
    """An uninitialised contiguous tensor of t's shape and device."""
    import torch
    if t.is_contiguous():
        return torch.empty_like(t, dtype=dtype)
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _strides(*tensors):
    """The strides argument: None where all are contiguous."""
    if all([t.is_contiguous() for t in tensors]):
        return None
    flat = [st for t in tensors for st in t.stride()[:3]]
    return (ctypes.c_longlong * len(flat))(*flat)


def _block_count(Sk, block):
    if block < 64 or block % 64:
        raise ValueError(f"block must be a positive multiple of 64, not {block}")
    if block > 1 << 30 or Sk > 1 << 30:  # more would not pass the C entry points' int whole
        raise ValueError(f"{Sk} keys in blocks of {block}: more than 2^30")
    return -(-Sk // block)


def dash_block_means(k, block, kv_len=None, start=None, out=None, stream=None):
    """fp32 means [B,Hkv,nb,D] of the key blocks of k [B,Hkv,Sk,D] (zeros for a block that
    has no keys below kv_len).  With `start` (int32 [B]) only the blocks from start[b] //
    block to the last one with keys are written into `out`, the others stay as they are."""
    import torch
    if k.dim() != 4:
        raise ValueError("k must be [B,Hkv,Sk,D]")
    B, Hkv, Sk, D = k.shape
    strides, device = _expect_input("k", k), k.device
    nb = _block_count(Sk, block)
    if start is not None and out is None:
        raise ValueError("start updates means in place: give them as out")
    n, s = _expect_rows("kv_len", kv_len, B, device), _expect_rows("start", start, B, device)
    if out is not None:
        _expect("out", out, (B, Hkv, nb, D), torch.float32, device)
    with _Launch(device, stream) as st:
        if out is None:
            out = k.new_empty((B, Hkv, nb, D), dtype=torch.float32)
        _check(load().dash_block_means(k.data_ptr(), strides, out.data_ptr(), n, s, B, Hkv, Sk,
                                       D, block, st), "dash_block_means")
    return out


def dash_block_select(q, means, seq_k, block, topk, causal=True, sink=1, local=1, kv_len=None,
                      q_start=None, out=None, stream=None):
    """The blocks each query attends to, int32 [B,Hkv,Sq,topk], ascending, then -1.  q
    [B,H,Sq,D]; means [B,Hkv,nb,D] of seq_k keys in blocks of `block`.  The first `sink` and
    the last `local` visible blocks are always among them."""
    import torch
    if q.dim() != 4 or means.dim() != 4:
        raise ValueError("q must be [B,H,Sq,D] and means [B,Hkv,nb,D]")
    B, H, Sq, D = q.shape
    Hkv = means.shape[1]
    if not (0 < topk <= 1 << 20 and 0 <= sink <= topk and 0 <= local <= topk - sink):
        raise ValueError(f"topk = {topk}, sink = {sink}, local = {local}: sink + local <= topk, "
                         "1 <= topk <= 2^20 are needed")
    strides, device = _expect_input("q", q), q.device
    _expect("means", means, (B, Hkv, _block_count(seq_k, block), D), torch.float32, device)
    n, s = _expect_rows("kv_len", kv_len, B, device), _expect_rows("q_start", q_start, B, device)
    if out is not None:
        _expect("out", out, (B, Hkv, Sq, topk), torch.int32, device)
    with _Launch(device, stream) as st:
        if out is None:
            out = q.new_empty((B, Hkv, Sq, topk), dtype=torch.int32)
        _check(load().dash_block_select(q.data_ptr(), strides, means.data_ptr(), out.data_ptr(),
                                        n, s, B, H, Hkv, Sq, seq_k, D, block, topk,
                                        int(bool(causal)), sink, local, st), "dash_block_select")
    return out


class SparsePlan:
    """A selection prepared by dash_sparse_plan for the forward and the backward."""
    __slots__ = ("buf", "shape", "causal", "stream", "has_kv_len", "has_q_start")

    def __init__(self, buf, shape, causal, stream, has_kv_len=True, has_q_start=True):
        self.buf, self.shape, self.causal = buf, shape, causal  # shape: B,H,Hkv,Sq,Sk,block,topk
        self.stream = stream  # handle of the stream the plan was made on
        self.has_kv_len, self.has_q_start = has_kv_len, has_q_start  # given when it was made

    def on(self, stream):
        """The plan's address for work on `stream` (a handle); the memory outlives that work."""
        if stream != self.stream:
            import torch
            self.buf.record_stream(torch.cuda.current_stream(self.buf.device))
        return self.buf.data_ptr()


def _bytes(n, what):
    if n < 0:
        raise DashError(int(-n), what)
    return int(n)


def dash_sparse_plan(idx, heads, seq_k, block, causal=True, kv_len=None, q_start=None, stream=None):
    """The plan of a selection idx (int32 [B,Hkv,Sq,topk]) for `heads` query heads and seq_k
    keys.  idx, kv_len and q_start are read by the call, not kept."""
    import torch
    if idx.dim() != 4:
        raise ValueError("idx must be [B,Hkv,Sq,topk]")
    B, Hkv, Sq, topk = idx.shape
    _expect("idx", idx, idx.shape, torch.int32)
    n = _expect_rows("kv_len", kv_len, B, idx.device)
    s = _expect_rows("q_start", q_start, B, idx.device)
    shape = (B, int(heads), Hkv, Sq, int(seq_k), int(block), topk)
    _block_count(*shape[4:6])
    if not 0 <= shape[1] < 1 << 31:
        raise ValueError(f"heads must be a number of query heads, not {heads}")
    lib = load()
    size = _bytes(lib.dash_sparse_plan_bytes(*shape), "dash_sparse_plan")
    with _Launch(idx.device, stream) as st:
        buf = idx.new_empty((max(size, 16),), dtype=torch.uint8)
        _check(lib.dash_sparse_plan(idx.data_ptr(), n, s, buf.data_ptr(), *shape, int(bool(causal)),
                                    st), "dash_sparse_plan")
    return SparsePlan(buf, shape, bool(causal), st, kv_len is not None, q_start is not None)


def _expect_qkv(q, k, v):
    """B, H, Hkv, Sq, Sk, D and the strides argument of q, k, v."""
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,Sq,D] and k [B,Hkv,Sk,D]")
    B, H, Sq, D = q.shape
    Bk, Hkv, Sk, Dk = k.shape
    bf, device = torch.bfloat16, q.device
    # the usual case at once: what is wrong is looked for only where something is
    if (Bk == B and Dk == D and v.shape == k.shape and q.dtype is bf and k.dtype is bf
            and v.dtype is bf and q.is_cuda and k.device == device and v.device == device
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
            and not (q.data_ptr() | k.data_ptr() | v.data_ptr()) & 15):
        return B, H, Hkv, Sq, Sk, D, None
    _expect("q", q, q.shape, bf, contiguous=False)
    _expect("k", k, (B, Hkv, Sk, D), bf, device, contiguous=False)
    _expect("v", v, k.shape, bf, device, contiguous=False)
    return B, H, Hkv, Sq, Sk, D, _strides(q, k, v)


def _expect_plan(plan, shape, device):
    if plan.shape[:5] != shape:
        raise ValueError(f"the plan is for B, H, Hkv, Sq, Sk = {plan.shape[:5]}, not {shape}")
    if plan.buf.device != device:
        raise ValueError(f"the plan must be on {device}")


def _expect_same_selection(plan, idx, block, causal, kv_len, q_start):
    """Reject a forward whose own arguments are not those of its plan, as far as they can be told
    without reading the device."""
    if block != plan.shape[5]:
        raise ValueError(f"the plan is for blocks of {plan.shape[5]}, not {block}")
    if causal is not None and bool(causal) != plan.causal:
        raise ValueError(f"the plan was made with causal = {plan.causal}")
    if idx is not None:
        B, _, Hkv, Sq, _, _, topk = plan.shape
        if idx.shape != (B, Hkv, Sq, topk):
            raise ValueError(f"idx has shape {tuple(idx.shape)}, the plan is for {(B, Hkv, Sq, topk)}")
    if kv_len is not None and not plan.has_kv_len:
        raise ValueError("the plan was made without kv_len")
    if q_start is not None and not plan.has_q_start:
        raise ValueError("the plan was made without q_start")


def _scale(scale):
    """The C calls' scale: None is their 0, 1 / sqrt(D).  A number that is 0 there would be taken
    for it."""
    if scale is None:
        return 0.0
    if ctypes.c_float(scale).value == 0.0:
        raise ValueError(f"scale must be positive, not {scale} (None is 1 / sqrt(D))")
    return float(scale)


def _few_queries(B, H, Hkv, Sq):
    """Whether each query reads its keys for itself, without a plan: single tokens, and short
    runs while a token of a K/V head (16 query heads at a time) leaves most SMs free.  Measured
    on 16 picks of 64 keys, 32 query and 8 K/V heads, D = 128, whole calls: 16 queries of one
    sequence take 19 us (34 with a plan), 32 take 25 (35); one token of 64 sequences takes 54 (53,
    and two more launches), two take 97 (74).  The rule does not look at the picks, and long
    ones are better off with a plan, which can be given: 16 queries of 4096 keys each take 44
    (35), of 16384 keys 138 (58); single tokens of 4096 and 16384 keys take the same either
    way."""
    return Sq == 1 or B * Hkv * Sq * -(-(H // max(Hkv, 1)) // 16) <= 256


def dash_attn_sparse_fwd(q, k, v, idx, block, causal=None, kv_len=None, q_start=None, scale=None,
                         plan=None, out=None, lse=None, stream=None):
    """O, LSE of attention over the selected blocks: q [B,H,Sq,D], k and v [B,Hkv,Sk,D] (any
    strides with a contiguous last dimension), idx int32 [B,Hkv,Sq,topk].  A query that sees
    nothing gets O = 0 and LSE = -inf.  causal: True unless given, or the plan's.  Give the
    `plan` of idx where the backward follows: the selection is then the plan's; block, and what
    else is given of idx, causal, kv_len and q_start, have to be those it was made with (the
    tensors' contents are not compared)."""
    import torch
    B, H, Hkv, Sq, Sk, D, strides = _expect_qkv(q, k, v)
    if out is not None:
        _expect("out", out, (B, H, Sq, D), torch.bfloat16, q.device)
    if lse is not None:
        _expect("lse", lse, (B, H, Sq), torch.float32, q.device)
    if plan is not None:
        _expect_same_selection(plan, idx, block, causal, kv_len, q_start)
    else:
        causal = causal is None or bool(causal)
        _expect("idx", idx, (B, Hkv, Sq, idx.shape[-1]), torch.int32, q.device)
        topk, blocks = idx.shape[-1], _block_count(Sk, block)
        if _few_queries(B, H, Hkv, Sq) and topk <= 1024 and blocks <= 65536:
            n = s = None
            if kv_len is not None:
                n = _expect_rows("kv_len", kv_len, B, q.device)
            if q_start is not None:
                s = _expect_rows("q_start", q_start, B, q.device)
            with _Launch(q.device, stream) as st:
                if out is None:
                    out = _like(q)
                if lse is None:
                    lse = q.new_empty((B, H, Sq), dtype=torch.float32)
                _check(load().dash_attn_sparse_tokens(
                    q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, idx.data_ptr(), n, s,
                    out.data_ptr(), lse.data_ptr(), B, H, Hkv, Sq, Sk, D, block, topk,
                    int(causal), _scale(scale), st), "dash_attn_sparse_fwd")
            return out, lse
        plan = dash_sparse_plan(idx, H, Sk, block, causal, kv_len, q_start, stream)
    _expect_plan(plan, (B, H, Hkv, Sq, Sk), q.device)
    lib = load()
    size = _bytes(lib.dash_attn_sparse_work_bytes(*plan.shape[:5], D, *plan.shape[5:], 0),
                  "dash_attn_sparse_fwd")
    with _Launch(q.device, stream) as st:
        if out is None:
            out = _like(q)
        if lse is None:
            lse = q.new_empty((B, H, Sq), dtype=torch.float32)
        work = q.new_empty((size,), dtype=torch.uint8) if size else None
        _check(lib.dash_attn_sparse_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        strides, plan.on(st), out.data_ptr(),
                                        lse.data_ptr(), work.data_ptr() if size else None,
                                        *plan.shape[:5], D, *plan.shape[5:], int(plan.causal),
                                        _scale(scale), st), "dash_attn_sparse_fwd")
    return out, lse


def dash_attn_sparse_bwd(q, k, v, o, do, lse, plan, scale=None, dq=None, dk=None, dv=None,
                         stream=None):
    """dQ [B,H,Sq,D], dK and dV [B,Hkv,Sk,D] of dash_attn_sparse_fwd with the same plan, from
    its O and LSE; bitwise reproducible."""
    import torch
    B, H, Hkv, Sq, Sk, D, _ = _expect_qkv(q, k, v)
    _expect("o", o, q.shape, torch.bfloat16, q.device)
    _expect("do", do, q.shape, torch.bfloat16, q.device, contiguous=False)
    _expect("lse", lse, (B, H, Sq), torch.float32, q.device)
    for name, t, shape in (("dq", dq, q.shape), ("dk", dk, k.shape), ("dv", dv, k.shape)):
        if t is not None:
            _expect(name, t, shape, torch.bfloat16, q.device)
    _expect_plan(plan, (B, H, Hkv, Sq, Sk), q.device)
    lib = load()
    size = _bytes(lib.dash_attn_sparse_work_bytes(*plan.shape[:5], D, *plan.shape[5:], 1),
                  "dash_attn_sparse_bwd")
    with _Launch(q.device, stream) as st:
        dq = _like(q) if dq is None else dq
        dk = _like(k) if dk is None else dk
        dv = _like(k) if dv is None else dv
        if H == 0:  # no head reads a key; the C call has nothing to do
            return dq, dk.zero_(), dv.zero_()
        work = q.new_empty((max(size, 16),), dtype=torch.uint8)
        _check(lib.dash_attn_sparse_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
                                        _strides(q, k, v, do), plan.on(st), o.data_ptr(),
                                        lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                        dv.data_ptr(), work.data_ptr(), *plan.shape[:5], D,
                                        *plan.shape[5:], int(plan.causal), _scale(scale), st),
               "dash_attn_sparse_bwd")
    return dq, dk, dv


# ---------------------------------------------------------------- 8-bit checkpoints
_LONGS = [ctypes.c_longlong * (4 * n) for n in range(5)]  # arguments of a launch of n tensors


def _check_ckpt(what, x, dtype, device):
    """x: contiguous device tensor of dtype in whole groups of 32, 16-byte aligned."""
    if (x.dtype is dtype and x.is_cuda and x.device == device and x.is_contiguous() and x.dim()
            and not x.shape[-1] % 32 and not x.data_ptr() % 16):
        return
    _expect(what, x, x.shape, dtype, device)
    raise ValueError(f"{what}: the last dimension must be a multiple of 32, 16-byte aligned")


def _ckpt_launch(call, what, inputs, exps, outputs, st):
    """Launches of up to four tensors: addresses and element counts in one argument array."""
    for a in range(0, len(inputs), 4):
        part = inputs[a:a + 4]
        n = len(part)
        args = _LONGS[n](*[x.data_ptr() for x in part], *[x.data_ptr() for x in exps[a:a + 4]],
                         *[x.data_ptr() for x in outputs[a:a + 4]], *[x.numel() for x in part])
        at = [ctypes.byref(args, 8 * n * k) for k in range(4)]
        if call == "pack":
            _check(load().dash_ckpt8_pack(at[0], at[2], at[1], at[3], n, st), what)
        else:
            _check(load().dash_ckpt8_unpack(at[0], at[1], at[2], at[3], n, st), what)


def dash_ckpt8_pack(*tensors, stream=None):
    """8-bit checkpoints of bf16 tensors (contiguous, last dimension a multiple of 32): for
    each a pair (m, e), int8 of the tensor's shape and int8 [..., D // 32]."""
    import torch
    if not tensors:
        return []
    device = tensors[0].device
    for x in tensors:
        _check_ckpt("the tensor", x, torch.bfloat16, device)
    with _Launch(device, stream) as st:
        ms = [torch.empty_like(x, dtype=torch.int8) for x in tensors]
        es = [x.new_empty((*x.shape[:-1], x.shape[-1] // 32), dtype=torch.int8) for x in tensors]
        _ckpt_launch("pack", "dash_ckpt8_pack", tensors, es, ms, st)
    return list(zip(ms, es))


def dash_ckpt8_unpack(*pairs, stream=None):
    """The bf16 tensors that checkpoints (m, e) stand for, exactly."""
    import torch
    if not pairs:
        return []
    device = pairs[0][0].device
    for m, e in pairs:
        _check_ckpt("m of a checkpoint", m, torch.int8, device)
        _expect("e of a checkpoint", e, (*m.shape[:-1], m.shape[-1] // 32), torch.int8, device)
    with _Launch(device, stream) as st:
        ms = [m for m, _ in pairs]
        out = [torch.empty_like(m, dtype=torch.bfloat16) for m in ms]
        _ckpt_launch("unpack", "dash_ckpt8_unpack", ms, [e for _, e in pairs], out, st)
    return out


def dash_attn_bwd_ckpt8(q8, k8, v8, o8, do, lse, causal: bool, schedule="shift", dq=None, dk=None,
                        dv=None, stream=None):
    """dash_attn_bwd (grouped-query where K/V have fewer heads) from the 8-bit checkpoints
    (m, e) of Q, K, V and O: the result is bitwise that of the backward on the values the
    checkpoints stand for."""
    import torch
    import contextlib
    ctx = torch.cuda.device(do.device) if stream is None else torch.cuda.stream(stream)
    with ctx if do.is_cuda else contextlib.nullcontext():
        q, k, v, o = dash_ckpt8_unpack(q8, k8, v8, o8, stream=stream)
        bwd = dash_attn_bwd if q.shape[1:2] == k.shape[1:2] else dash_attn_bwd_gqa
        return bwd(q, k, v, o, do, lse, causal, schedule, dq, dk, dv, stream)


def dash_attn_sparse_bwd_ckpt8(q8, k8, v8, o8, do, lse, plan, scale=None, dq=None, dk=None,
                               dv=None, stream=None):
    """dash_attn_sparse_bwd from the 8-bit checkpoints of Q, K, V and O."""
    q, k, v, o = dash_ckpt8_unpack(q8, k8, v8, o8, stream=stream)
    return dash_attn_sparse_bwd(q, k, v, o, do, lse, plan, scale, dq, dk, dv, stream)
