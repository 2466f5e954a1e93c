"""Windowed attention with sinks, received key weights and cache eviction: plans and refusals (CPU only)."""
import ctypes

import pytest
import torch

import mla_paged_decode_04_b200 as mla
from mla_paged_decode_04_b200 import _lib

FAKE = 1 << 20  # 256-byte aligned, never dereferenced: every call here is refused on the host
vp = ctypes.c_void_p


def test_sinks_live_on_the_plan_beside_the_window():
    p = mla.mla_decode_plan(2, 4, 32, 1000, "fp8")
    size = p.workspace_bytes
    assert p.sinks == 0
    assert mla.mla_decode_plan_sinks(p, 7) is p and p.sinks == 7 and p.window == 0
    mla.mla_decode_plan_window(p, 100)
    assert p.sinks == 7 and p.window == 100 and p.workspace_bytes == size
    mla.mla_decode_plan_sinks(p, 0)
    assert p.sinks == 0 and p.window == 100
    assert mla.mla_decode_plan(2, 4, 32, 1000, "fp8").sinks == 0  # plans are remembered without it
    for plan in (mla.mla_prefill_plan(2, 9, 32, 1000, "bf16"), mla.mla_decode_plan_custom(2, 4, 32, 1000, "fp8",
                                                                                           kernel="simt")):
        assert mla.mla_decode_plan_sinks(plan, 3).sinks == 3


def test_sinks_are_refused_where_a_window_is():
    lib = _lib.lib()
    p = mla.mla_decode_plan(2, 4, 32, 1000, "fp8")
    assert lib.mla_decode_plan_sinks(None, 1) == -1
    assert lib.mla_decode_plan_sinks(ctypes.byref(p), -1) == -1
    solo = mla.mla_decode_plan_custom(2, 4, 32, 1000, "fp8", kernel="tcgen05_solo")
    with pytest.raises(mla.MlaError) as e:
        mla.mla_decode_plan_sinks(solo, 1)
    assert e.value.code == -2
    many = mla.mla_decode_plan(20000, 1, 16, 64, "bf16")  # fixed splits: more units than the balanced schedule takes
    assert lib.mla_decode_plan_sinks(ctypes.byref(many), 1) == -2
    assert lib.mla_decode_plan_sinks(ctypes.byref(many), 0) == 0
    bad = _lib.MlaPlan.from_buffer_copy(p)
    bad.magic = 0
    assert lib.mla_decode_plan_sinks(ctypes.byref(bad), 1) == -6
    bad = _lib.MlaPlan.from_buffer_copy(p)
    bad.sinks = -1
    assert weights_call(bad) == -6


def weights_call(plan, **kw):
    a = dict(q=FAKE, total_q=8, cu=0, kv=FAKE, pages=8, page_size=64, bt=FAKE, maxp=16, sl=FAKE, scale=0.04, qs=1.0,
             ks=1.0, lse=FAKE, w_in=FAKE, in_stride=1024, decay=1.0, w_out=FAKE, out_stride=1024, cols=1024,
             status=FAKE)
    a.update(kw)
    return _lib.lib().mla_key_weights(
        ctypes.byref(plan) if plan is not None else None, vp(a["q"]), a["total_q"], vp(a["cu"]), vp(a["kv"]),
        a["pages"], a["page_size"], vp(a["bt"]), a["maxp"], vp(a["sl"]), a["scale"], a["qs"], a["ks"], vp(a["lse"]),
        vp(a["w_in"]), a["in_stride"], a["decay"], vp(a["w_out"]), a["out_stride"], a["cols"], vp(a["status"]), None)


def test_key_weights_refuses_bad_arguments_before_any_launch():
    p = mla.mla_decode_plan(2, 4, 32, 1000, "fp8")
    assert weights_call(None) == -6
    for name in ("q", "kv", "bt", "sl", "lse", "w_out", "status"):
        assert weights_call(p, **{name: 0}) == -1, name
    for name in ("q", "kv"):
        assert weights_call(p, **{name: FAKE + 8}) == -1, name
    for name in ("bt", "sl", "lse", "w_in", "w_out", "status"):
        assert weights_call(p, **{name: FAKE + 2}) == -1, name
    inf, nan = float("inf"), float("nan")
    for kw in (dict(pages=0), dict(maxp=0), dict(scale=inf), dict(scale=nan), dict(decay=nan), dict(decay=inf),
               dict(decay=-0.5), dict(qs=0.0), dict(ks=nan), dict(cols=999), dict(out_stride=1023),
               dict(in_stride=1023), dict(cols=2000),
               dict(w_in=FAKE + 4), dict(w_in=FAKE + 4 * 1023), dict(w_in=FAKE, in_stride=1025),  # shifted in place
               dict(w_in=FAKE + 4 * 500, in_stride=1500, out_stride=1500)):
        assert weights_call(p, **kw) == -1, kw
    assert weights_call(p, page_size=32) == -2
    assert weights_call(p, pages=(1 << 25) + 1) == -2
    assert weights_call(p, cu=FAKE) == -6            # ragged offsets with a decode plan
    r = mla.mla_prefill_plan(2, 9, 32, 1000, "bf16")
    assert weights_call(r) == -1                     # a prefill plan without them
    assert weights_call(r, cu=FAKE, total_q=19) == -1
    assert weights_call(r, cu=FAKE, total_q=-1) == -1
    assert weights_call(mla.mla_decode_plan(0, 4, 32, 1000, "fp8"), q=0, kv=0) == 0  # an empty batch


def test_weights_may_lie_beside_each_other_in_one_buffer():
    """Column slices of one buffer do not overlap; the call gets past that check (and ends at the host pointers)."""
    p = mla.mla_decode_plan(2, 4, 32, 1000, "fp8")
    code = weights_call(p, w_in=FAKE + 4 * 1024, in_stride=2048, out_stride=2048)
    assert code in (-1, -4, -5) and code == weights_call(p)
    assert weights_call(p, w_in=FAKE + 4 * 1023, in_stride=2048, out_stride=2048) == -1


def evict_call(**kw):
    a = dict(w=FAKE, w_stride=1000, cols=1000, sl=FAKE, batch=2, budget=128, sinks=4, recent=32, kv=FAKE, pages=8,
             page_size=64, bt=FAKE, maxp=16, out=2 * FAKE, out_pages=8, out_bt=2 * FAKE, out_maxp=2, dtype=0,
             out_sl=FAKE, kept=FAKE, out_w=0, out_w_stride=128, status=0)
    a.update(kw)
    return _lib.lib().mla_cache_evict(
        vp(a["w"]), a["w_stride"], a["cols"], vp(a["sl"]), a["batch"], a["budget"], a["sinks"], a["recent"],
        vp(a["kv"]), a["pages"], a["page_size"], vp(a["bt"]), a["maxp"], vp(a["out"]), a["out_pages"],
        vp(a["out_bt"]), a["out_maxp"], a["dtype"], vp(a["out_sl"]), vp(a["kept"]), vp(a["out_w"]),
        a["out_w_stride"], vp(a["status"]), None)


def test_cache_evict_refuses_bad_arguments_before_any_launch():
    for name in ("w", "sl", "kv", "bt", "out", "out_bt", "out_sl", "kept"):
        assert evict_call(**{name: 0}) == -1, name
    for name in ("kv", "out"):
        assert evict_call(**{name: 3 * FAKE + 8}) == -1, name
    for name in ("w", "sl", "bt", "out_bt", "out_sl", "kept", "out_w", "status"):
        assert evict_call(**{name: 3 * FAKE + 2}) == -1, name
    for kw in (dict(batch=-1), dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=100, recent=29),
               dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), dict(pages=0), dict(out_pages=0), dict(maxp=0),
               dict(cols=0), dict(w_stride=999), dict(out_maxp=1), dict(dtype=3),
               dict(out=FAKE, out_bt=FAKE),                       # onto its own pages
               dict(out_w=FAKE + 400), dict(out_w=9 * FAKE, out_w_stride=127)):
        assert evict_call(**kw) == -1, kw
    assert evict_call(page_size=16) == -2
    # places of keys are ints: no more than 2^30 of them, where columns and table both allow more
    many = (1 << 30) // 64
    assert evict_call(cols=(1 << 30) + 1, w_stride=(1 << 30) + 1, maxp=many + 1) == -2
    assert evict_call(budget=(1 << 30) + 1, out_maxp=many + 1) == -2
    assert evict_call(batch=0) == 0


def test_bindings_refuse_what_the_library_cannot_see():
    p = mla.mla_decode_plan(1, 1, 16, 64, "bf16")
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mla.key_weights(p, q, q, q, q, 1.0, q, q, q)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.cache_evict(torch.zeros(1, 64), lens, q, lens, q, lens, 4)
