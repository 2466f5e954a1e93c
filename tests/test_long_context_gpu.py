"""Windowed attention with sinks, received key weights and cache eviction on the GPU, against plain 64-bit forms.
The bounds come from the roundings each path makes (long_context_ref.py)."""
import math
import types

import pytest
import torch

import long_context_ref as ref
import mla_paged_decode_04_b200 as mla
from mla_paged_decode_04_b200 import _lib
from mla_paged_decode_04_b200.inputs import make_inputs_custom, make_prefill_inputs

pytestmark = pytest.mark.gpu
KERNELS = ["simt", "auto"]


def decode(g, window, sinks, kernel="auto", **kw):
    dec = mla.MlaDecoder(g.batch, g.q_len, g.heads, max(g.max_seq_len, 1), g.dtype, g.q.device, kernel=kernel,
                         window=window, sinks=sinks, **kw)
    out, lse = dec(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale)
    return dec, out, lse


def prefill(g, window, sinks, kernel="auto"):
    pre = mla.MlaPrefill(g.batch, g.max_q_len, g.heads, max(g.max_seq_len, 1), g.dtype, g.q.device, kernel=kernel,
                         window=window, sinks=sinks)
    out, lse = pre(g.q, g.cu_seqlens_q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale,
                   g.kv_scale)
    return pre, out, lse


def check_attention(g, out, lse, window, sinks, kernel, what):
    o, l, tol, ltol = ref.attention(g, window, sinks, p_step=0.0 if kernel == "simt" else None)
    ref.close(out.reshape(o.shape), o, tol, what + " out")
    ref.close(lse.reshape(l.shape), l, ltol, what + " lse")


# (B, T, H, dtype, seq_lens, window, sinks)
WINDOWED = [
    (1, 1, 16, "bf16", [600], 100, 4),
    (1, 1, 1, "fp16", [700], 64, 1),                   # one row
    (2, 4, 32, "fp8", [1000, 77], 128, 4),
    (3, 4, 16, "fp16", [64, 65, 300], 1, 1),           # a window of one key
    (3, 2, 128, "bf16", [700, 3, 0], 33, 70),          # more sinks than window, two pages of sinks; empty entry
    (3, 4, 33, "fp8", [2, 640, 641], 200, 128),        # seq_len < q_len; sinks end on a pair of pages
    (2, 3, 40, "fp8", [515, 130], 256, 129),           # sinks one key into a third page
    (4, 1, 8, "bf16", [1, 2, 63, 64], 16, 5),
    (2, 4, 64, "fp16", [513, 1300], 300, 64),          # two query groups
    (2, 4, 64, "fp8", [513, 1300], 300, 63),
    (2, 2, 16, "bf16", [400, 200], 350, 100),          # window and sinks meet or cover everything
    (2, 2, 16, "fp8", [400, 200], 4000, 100),          # a window longer than every sequence
    (1, 2, 16, "bf16", [300], 40, 5000),               # sinks past the sequence
]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", range(len(WINDOWED)))
def test_windowed_decode_with_sinks(cuda_device, case, kernel):
    B, T, H, dt, lens, window, sinks = WINDOWED[case]
    g = make_inputs_custom(B, T, H, dt, lens, seed=300 + case, pool=2.0).to(cuda_device)
    dec, out, lse = decode(g, window, sinks, kernel)
    assert dec.status() == 0
    check_attention(g, out, lse, window, sinks, kernel, f"case {case}")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("new,prefix,window,sinks", [
    ([5, 0, 37, 1], [100, 30, 0, 700], 20, 4),
    ([130, 3], [250, 900], 128, 66),
])
def test_windowed_prefill_with_sinks(cuda_device, new, prefix, window, sinks, dtype, kernel):
    g = make_prefill_inputs(new, prefix, 24, dtype, seed=41).to(cuda_device)
    pre, out, lse = prefill(g, window, sinks, kernel)
    assert pre.status() == 0
    check_attention(g, out, lse, window, sinks, kernel, f"{dtype} {new}")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_sinks_without_effect_leave_every_bit(cuda_device, dtype):
    """No window: sinks change nothing; no sinks: the plain window."""
    g = make_inputs_custom(3, 2, 32, dtype, [500, 130, 1], seed=5, pool=1.5).to(cuda_device)
    for window, sinks in ((0, 7), (90, 0)):
        _, a, la = decode(g, window, sinks)
        _, b, lb = decode(g, window, 0)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["fp16", "fp8"])
def test_the_longest_window_with_fewer_keys_than_tokens(cuda_device, dtype, kernel):
    """A window of 2^31 - 1 stands for none, also where a row's last place is far below zero."""
    g = make_inputs_custom(4, 9, 20, dtype, [2, 0, 70, 9], seed=15, pool=1.5).to(cuda_device)
    for sinks in (0, 3):
        dec, out, lse = decode(g, (1 << 31) - 1, sinks, kernel)
        check_attention(g, out, lse, 0, 0, kernel, f"{sinks} sinks")
        got = dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse,
                              torch.zeros(4, 70, device=cuda_device), q_scale=g.q_scale, kv_scale=g.kv_scale)
        assert dec.status() == 0
        want, tol = ref.key_weights(g, lse.reshape(-1, 20), None, 1.0, 70)
        ref.close(got, want, tol, f"{sinks} sinks, weights")


def poisoned(g, window, sinks):
    """The same step with NaN in every place no row sees: the rest of the last page, the pages between sinks and
    window, whose table entries are -1, and page 0 of the pool where no entry owns it."""
    cache = g.kv_cache.clone()
    tables = g.block_tables.clone()
    flat = cache.view(torch.uint8).view(-1, 576 * cache.element_size())
    owned = set()
    new = g.cu_seqlens_q.diff().tolist() if hasattr(g, "cu_seqlens_q") else [g.q_len] * g.batch
    for b, n in enumerate(g.seq_lens.tolist()):
        pages = (n + 63) // 64
        seen = set()
        for t in range(new[b]):
            seen.update(ref.visible(n - new[b] + t + 1, window, sinks))
        for j in range(pages * 64):
            page = int(tables[b, j // 64])
            if j not in seen:
                flat[page * 64 + j % 64] = 0xFF  # a NaN in every type
        for i in range(pages):
            if any(i * 64 <= j < i * 64 + 64 for j in seen):
                owned.add(int(tables[b, i]))
            else:
                g_page = int(tables[b, i])
                flat[g_page * 64:(g_page + 1) * 64] = 0xFF
                tables[b, i] = -1
    for page in range(cache.shape[0]):
        if page not in owned:
            flat[page * 64:(page + 1) * 64] = 0xFF
    return cache, tables


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp8"])
def test_unseen_places_may_hold_nan_and_their_pages_may_be_gone(cuda_device, dtype, kernel):
    window, sinks = 70, 5
    g = make_inputs_custom(3, 2, 32, dtype, [1000, 391, 130], seed=9, pool=2.0).to(cuda_device)
    _, want, want_l = decode(g, window, sinks, kernel)
    cache, tables = poisoned(g, window, sinks)
    dec = mla.MlaDecoder(3, 2, 32, 1000, dtype, cuda_device, kernel=kernel, window=window, sinks=sinks)
    for _ in range(2):
        out, lse = dec(g.q, cache, tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale)
        assert dec.status() == 0
        assert torch.equal(out, want) and torch.equal(lse, want_l)


# (B, T, H, dtype, seq_lens, window, sinks)
WEIGHED = [
    (1, 1, 16, "bf16", [600], 0, 0),
    (1, 1, 1, "fp16", [1], 0, 0),
    (2, 4, 32, "fp8", [1000, 77], 0, 0),
    (3, 2, 128, "bf16", [700, 3, 0], 0, 0),            # 256 rows; an empty entry
    (3, 4, 33, "fp8", [2, 640, 641], 100, 7),          # 132 rows; seq_len < q_len
    (2, 3, 100, "fp16", [515, 256], 0, 0),             # 300 rows: more than one group of 256
    (2, 5, 128, "bf16", [513, 300], 37, 70),
    (2, 5, 128, "fp8", [1025, 257], 600, 3),
    (4, 1, 5, "fp8", [1, 63, 64, 65], 0, 0),
    (130, 1, 16, "fp8", [(37 * i) % 300 for i in range(130)], 0, 0),
]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", range(len(WEIGHED)))
def test_key_weights_of_a_decode_step(cuda_device, case, kernel):
    B, T, H, dt, lens, window, sinks = WEIGHED[case]
    g = make_inputs_custom(B, T, H, dt, lens, seed=500 + case, pool=2.0).to(cuda_device)
    dec, _, lse = decode(g, window, sinks, kernel)
    cols = g.max_seq_len + 3
    before = torch.rand(B, cols, generator=torch.Generator().manual_seed(case)).to(cuda_device)
    for decay in (1.0, 0.25):
        after = torch.full((B, cols), -7.0, device=cuda_device)
        got = dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse, after,
                              weights=before, decay=decay, q_scale=g.q_scale, kv_scale=g.kv_scale)
        assert got is after and dec.status() == 0
        want, tol = ref.key_weights(g, lse.reshape(-1, H), before, decay, cols, window, sinks)
        past = torch.arange(cols, device=cuda_device)[None] >= g.seq_lens[:, None]
        assert (after[past] == -7.0).all()
        ref.close(torch.where(past, 0.0, after), want, tol, f"case {case} decay {decay}")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("new,prefix,heads,window,sinks", [
    ([5, 0, 37, 1], [100, 30, 0, 700], 24, 0, 0),
    ([130, 3, 64], [250, 900, 1], 20, 0, 0),
    ([40, 70], [600, 333], 128, 90, 66),
])
def test_key_weights_of_a_ragged_step(cuda_device, new, prefix, heads, window, sinks, dtype, kernel):
    g = make_prefill_inputs(new, prefix, heads, dtype, seed=43).to(cuda_device)
    pre, _, lse = prefill(g, window, sinks, kernel)
    after = torch.zeros(g.batch, g.max_seq_len, device=cuda_device)
    pre.key_weights(g.q, g.cu_seqlens_q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse, after,
                    q_scale=g.q_scale, kv_scale=g.kv_scale)
    assert pre.status() == 0
    want, tol = ref.key_weights(g, lse, None, 1.0, g.max_seq_len, window, sinks)
    ref.close(after, want, tol, f"{dtype} {new}")


@pytest.mark.parametrize("kernel", KERNELS)
def test_weights_of_a_full_step_sum_to_the_rows(cuda_device, kernel):
    g = make_inputs_custom(3, 4, 32, "bf16", [900, 130, 4], seed=3, pool=1.5).to(cuda_device)
    dec, _, lse = decode(g, 0, 0, kernel)
    w = torch.zeros(3, 900, device=cuda_device)
    dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse, w)
    assert (w.double().sum(1) - 128.0).abs().max() < 128 * 1e-4


@pytest.mark.parametrize("kernel", KERNELS)
def test_key_weights_in_place_strided_and_repeatable(cuda_device, kernel):
    g = make_inputs_custom(2, 2, 128, "fp8", [700, 333], seed=4, pool=1.5).to(cuda_device)
    dec, _, lse = decode(g, 0, 0, kernel)
    args = (g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse)
    kw = dict(q_scale=g.q_scale, kv_scale=g.kv_scale)
    one = dec.key_weights(*args, torch.zeros(2, 700, device=cuda_device), **kw)
    wide = torch.full((2, 1000), 3.0, device=cuda_device)
    view = wide[:, 100:800]
    dec.key_weights(*args, view, weights=None, **kw)
    assert torch.equal(view[0], one[0]) and torch.equal(view[1, :333], one[1, :333])
    assert (wide[:, :100] == 3.0).all() and (wide[:, 800:] == 3.0).all() and (view[1, 333:] == 3.0).all()
    acc = one.clone()
    dec.key_weights(*args, acc, weights=acc, decay=1.0, **kw)
    assert torch.equal(acc, one * 2)
    # decay 0 does not read the old weights
    dec.key_weights(*args, acc.fill_(math.nan), weights=acc, decay=0.0, **kw)
    assert torch.equal(acc[0], one[0]) and torch.equal(acc[1, :333], one[1, :333])


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_key_weights_pass_over_unseen_places(cuda_device, dtype, kernel):
    window, sinks = 70, 5
    g = make_inputs_custom(3, 2, 32, dtype, [1000, 391, 130], seed=9, pool=2.0).to(cuda_device)
    dec, _, lse = decode(g, window, sinks, kernel)
    kw = dict(q_scale=g.q_scale, kv_scale=g.kv_scale)
    w0 = torch.rand(3, 1000, device=cuda_device)
    want = dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse, w0.clone(), weights=w0,
                           decay=0.5, **kw)
    cache, tables = poisoned(g, window, sinks)
    got = dec.key_weights(g.q, cache, tables, g.seq_lens, g.softmax_scale, lse, w0.clone(), weights=w0, decay=0.5,
                          **kw)
    assert dec.status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("kernel", KERNELS)
def test_key_weights_on_a_bad_page(cuda_device, kernel):
    g = make_inputs_custom(2, 1, 32, "bf16", [300, 200], seed=6, pool=1.5).to(cuda_device)
    dec, _, lse = decode(g, 0, 0, kernel)
    want = dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse,
                           torch.zeros(2, 300, device=cuda_device))
    assert dec.status() == 0
    tables = g.block_tables.clone()
    tables[0, 1], tables[1, 3] = -1, g.kv_cache.shape[0]
    got = dec.key_weights(g.q, g.kv_cache, tables, g.seq_lens, g.softmax_scale, lse,
                          torch.zeros(2, 300, device=cuda_device))
    assert dec.status() == mla.MLA_DEV_BAD_PAGE
    want[0, 64:128] = 0.0
    want[1, 192:200] = 0.0
    assert torch.equal(got, want)


def test_key_weights_without_new_tokens_only_decay(cuda_device):
    g = make_prefill_inputs([0, 0], [100, 30], 16, "bf16", seed=2).to(cuda_device)
    pre = mla.MlaPrefill(2, 4, 16, 100, "bf16", cuda_device)
    w = torch.rand(2, 100, device=cuda_device)
    got = pre.key_weights(g.q, g.cu_seqlens_q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale,
                          torch.empty(0, 16, device=cuda_device), torch.zeros_like(w), weights=w, decay=0.5)
    assert torch.equal(got[0], w[0] * 0.5) and torch.equal(got[1, :30], w[1, :30] * 0.5) and (got[1, 30:] == 0).all()


def test_key_weights_between_slices_of_one_buffer(cuda_device):
    g = make_inputs_custom(3, 1, 32, "bf16", [300, 100, 7], seed=8, pool=1.5).to(cuda_device)
    dec, _, lse = decode(g, 0, 0)
    args = (g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse)
    both = torch.rand(3, 600, device=cuda_device)
    old = both[:, 300:].clone()
    want = dec.key_weights(*args, both[:, :300].clone(), weights=old)
    dec.key_weights(*args, both[:, :300], weights=both[:, 300:])
    assert torch.equal(both[:, :300], want) and torch.equal(both[:, 300:], old)
    with pytest.raises(mla.MlaError) as e:
        dec.key_weights(*args, both[:, 1:301], weights=both[:, :300])
    assert e.value.code == -1


def test_key_weights_of_more_entries_than_one_launch_takes(cuda_device):
    """1024 entries' tile counts fit a launch's shared memory; the rest go to further launches."""
    lens = [(11 * i) % 90 for i in range(1500)]
    g = make_inputs_custom(1500, 1, 3, "fp8", lens, seed=12, pool=1.1).to(cuda_device)
    dec, _, lse = decode(g, 0, 0)
    after = torch.full((1500, 90), -1.0, device=cuda_device)
    dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse, after, q_scale=g.q_scale,
                    kv_scale=g.kv_scale)
    assert dec.status() == 0
    want, tol = ref.key_weights(g, lse.reshape(-1, 3), None, 1.0, 90)
    past = torch.arange(90, device=cuda_device)[None] >= g.seq_lens[:, None]
    assert (after[past] == -1.0).all()
    ref.close(torch.where(past, 0.0, after), want, tol, "1500 entries")


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_windowed_prefill_with_long_piece_lists(cuda_device, dtype):
    """One token per unit (65 heads): the pairs' lists go past the pieces whose geometry is kept (32) and past those
    in shared memory (64)."""
    new = [400] * 12 + [3, 0]
    g = make_prefill_inputs(new, [0, 5, 50, 64] * 3 + [700, 9], 65, dtype, seed=44, pool=1.2, device="cuda")
    g = g.to(cuda_device)
    pre, out, lse = prefill(g, 40, 3)
    assert pre.status() == 0
    check_attention(g, out, lse, 40, 3, "auto", dtype)


def test_sinks_at_full_sequence_length(cuda_device):
    """Pages far into a long sequence: 80,000 keys, of which a window and the sinks are read."""
    g = make_inputs_custom(2, 4, 32, "fp8", [80001, 79000], seed=77, pool=1.0, ).to(cuda_device)
    dec, out, lse = decode(g, 1500, 100)
    assert dec.status() == 0
    check_attention(g, out, lse, 1500, 100, "auto", "long")
    after = torch.zeros(2, 80001, device=cuda_device)
    dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse, after, q_scale=g.q_scale,
                    kv_scale=g.kv_scale)
    want, tol = ref.key_weights(g, lse.reshape(-1, 32), None, 1.0, 80001, 1500, 100)
    ref.close(after, want, tol, "long weights")


def test_a_wait_that_runs_out_with_sinks(cuda_device):
    """The FP8 pair kernel's failure-detection mode (its first tiles are never loaded, the waits for them end after
    their limit) on a plan with sinks; the next call is clean."""
    g = make_inputs_custom(2, 4, 32, "fp8", [3000, 1200], seed=62, pool=2.0).to(cuda_device)
    dec, out, lse = decode(g, 500, 4)
    faulty = type(dec.plan).from_buffer_copy(dec.plan)
    faulty.fault_test = 1
    mla.mla_decode(faulty, g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, out.clone(), lse.clone(),
                   dec.workspace, g.q_scale, g.kv_scale)
    torch.cuda.synchronize()
    assert dec.status() & mla.MLA_DEV_TIMEOUT
    again, lse2 = dec(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale)
    assert dec.status() == 0 and torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_sinks_through_the_bounds_checking_build(cuda_device, dtype, monkeypatch):
    monkeypatch.setattr(_lib, "_lib", _lib.load_library(_lib.CHECK_LIB_PATH))
    assert mla.bounds_checked()
    for lens, window, sinks in (([3000, 65, 1], 500, 4), ([1000, 391, 130], 70, 130)):
        g = make_inputs_custom(3, 4, 32, dtype, lens, seed=63, pool=2.0).to(cuda_device)
        dec, out, lse = decode(g, window, sinks)
        assert dec.status() == 0
        check_attention(g, out, lse, window, sinks, "auto", f"checking build {dtype}")
    g = make_prefill_inputs([3, 50, 1, 64], [100, 0, 4000, 63], 32, dtype, seed=201).to(cuda_device)
    pre, out, lse = prefill(g, 90, 65)
    assert pre.status() == 0
    check_attention(g, out, lse, 90, 65, "auto", f"checking build {dtype} prefill")


def evict_inputs(lens, dtype, budget, seed, device):
    """A cache of random bytes (rows move as they are, whatever they hold), its tables, and the pages to go to."""
    gen = torch.Generator(device=device).manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}[dtype]
    need = [(n + 63) // 64 for n in lens]
    pool = int(1.5 * sum(need)) + 1
    raw = torch.randint(0, 256, (pool, 64, 576 * dt.itemsize), generator=gen, device=device, dtype=torch.uint8)
    perm = torch.randperm(pool, generator=gen, device=device).to(torch.int32)
    tables = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device=device)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = perm[at:at + k]
        at += k
    g = types.SimpleNamespace(kv_cache=raw.view(dt), block_tables=tables,
                              seq_lens=torch.tensor(lens, dtype=torch.int32, device=device))
    per = (budget + 63) // 64
    pages = len(lens) * per + 3
    out_tables = torch.randperm(pages, generator=gen, device=device)[:len(lens) * per].to(torch.int32).view(-1, per)
    out_cache = torch.full((pages, 64, 576), 1.5, device=device).to(dt)
    return g, out_cache, out_tables


def check_evicted(g, weights, budget, sinks, recent, out_cache, out_tables, got):
    lens, kept, out_w = got
    raw = lambda c: c.view(torch.uint8).view(-1, 576 * c.element_size())  # noqa: E731
    src, dst = raw(g.kv_cache), raw(out_cache)
    mark = raw(torch.full((1, 1, 576), 1.5, device=dst.device).to(out_cache.dtype))[0]
    untouched = torch.ones(dst.shape[0], dtype=torch.bool, device=dst.device)
    for b, want in enumerate(ref.evict(weights, g.seq_lens.tolist(), budget, sinks, recent)):
        m = len(want)
        assert int(lens[b]) == m
        assert kept[b].tolist() == want + [-1] * (budget - m)
        j = torch.tensor(want, dtype=torch.long, device=dst.device)
        i = torch.arange(m, device=dst.device)
        to = out_tables[b].long()[i // 64] * 64 + i % 64
        frm = g.block_tables[b].long()[j // 64] * 64 + j % 64
        assert torch.equal(dst[to], src[frm])
        assert torch.equal(out_w[b, :m], weights[b, j]) or torch.isnan(weights[b, j]).any()
        untouched[to] = False
        rest = torch.arange(m, (m + 63) // 64 * 64, device=dst.device)
        at = out_tables[b].long()[rest // 64] * 64 + rest % 64
        assert (dst[at] == 0).all()  # the rest of the last page
        untouched[at] = False
    assert (dst[untouched] == mark).all()


EVICTIONS = [
    # lens, budget, sinks, recent
    ([1], 1, 0, 0),
    ([300, 64, 0, 65], 64, 4, 16),
    ([300, 129], 100, 0, 0),
    ([300, 129], 100, 60, 40),            # nothing left to choose
    ([1500, 700, 701, 2], 700, 7, 133),
    ([5000], 4000, 1, 1),
    ([4097, 33], 1, 0, 0),                # one key stays
    ([4097, 33], 1, 0, 1),
    ([40000, 17], 5000, 4, 64),
    ([(13 * i) % 200 for i in range(230)], 70, 3, 9),        # one CTA an entry that moves its rows too
    ([(131 * i) % 5000 for i in range(70)], 300, 3, 9),
    ([(331 * i) % 11000 for i in range(70)], 300, 3, 9),     # a cluster of four an entry that moves its rows too
    ([(331 * i) % 11000 for i in range(110)], 70, 3, 9),     # a cluster of two an entry
    ([10300, 9, 10240], 5000, 0, 1),                         # a cluster of eight
    ([10239] * 2, 5000, 0, 1),                               # the longest that one CTA takes
    ([400000], 600, 4, 100),                                  # a stretch longer than shared memory holds
]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(EVICTIONS)))
def test_evict(cuda_device, case, dtype):
    lens, budget, sinks, recent = EVICTIONS[case]
    g, out_cache, out_tables = evict_inputs(lens, dtype, budget, 70 + case, cuda_device)
    gen = torch.Generator().manual_seed(case)
    w = torch.exp(2 * torch.randn(len(lens), max(lens), generator=gen)).to(cuda_device)
    got = mla.cache_evict(w, g.seq_lens, g.kv_cache, g.block_tables, out_cache, out_tables, budget, sinks, recent)
    check_evicted(g, w, budget, sinks, recent, out_cache, out_tables, got)


@pytest.mark.parametrize("kind", ["equal", "few values", "signs", "nan", "inf", "tiny"])
def test_evict_orders_every_kind_of_weight(cuda_device, kind):
    lens, budget, sinks, recent = [1000, 777, 3000], 200, 3, 20
    g, out_cache, out_tables = evict_inputs(lens, "fp16", budget, 17, cuda_device)
    gen = torch.Generator().manual_seed(1)
    w = torch.randn(3, 3000, generator=gen)
    if kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "few values":
        w = torch.round(w * 2) / 2
    elif kind == "signs":
        w = torch.where(w > 0.5, 0.0, torch.where(w < -0.5, -0.0, w * 1e-3))
    elif kind == "nan":
        w = torch.where(w > -1.2, math.nan, w)
    elif kind == "inf":
        w = torch.where(w > 1, math.inf, torch.where(w < 0.9, -math.inf, w))
    else:
        w = w.abs() * 1e-41  # below the normal range
    w = w.to(cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = mla.cache_evict(w, g.seq_lens, g.kv_cache, g.block_tables, out_cache, out_tables, budget, sinks, recent,
                          device_status=status)
    check_evicted(g, w, budget, sinks, recent, out_cache, out_tables, got)
    assert int(status) == 0


def test_evict_within_one_pool_strided_weights_and_lengths_in_place(cuda_device):
    """The result on other pages of the same cache; weights as a slice; out_seq_lens = seq_lens."""
    lens, budget = [500, 90], 128
    g = make_inputs_custom(2, 1, 1, "bf16", lens, seed=21, pool=3.0).to(cuda_device)
    used = set(g.block_tables.flatten().tolist())
    free = [p for p in range(g.kv_cache.shape[0]) if p not in used][:4]
    out_tables = torch.tensor(free, dtype=torch.int32, device=cuda_device).view(2, 2)
    before = g.kv_cache.clone()
    wide = torch.rand(2, 900, device=cuda_device)
    w = wide[:, 33:533]
    seq = g.seq_lens.clone()
    new_w = torch.full((2, 200), -1.0, device=cuda_device)
    new, kept, out_w = mla.cache_evict(w, seq, g.kv_cache, g.block_tables, g.kv_cache, out_tables, budget, 4, 32,
                                       out_seq_lens=seq, out_weights=new_w)
    assert new is seq and seq.tolist() == [128, 90] and out_w is new_w
    want = ref.evict(w, lens, budget, 4, 32)
    for b in range(2):
        m = len(want[b])
        assert kept[b, :m].tolist() == want[b]
        i, j = torch.arange(m, device=cuda_device), torch.tensor(want[b], device=cuda_device)
        rows = g.kv_cache.view(-1, 576)[out_tables[b].long()[i // 64] * 64 + i % 64]
        assert torch.equal(rows, before.view(-1, 576)[g.block_tables[b].long()[j // 64] * 64 + j % 64])
        assert torch.equal(new_w[b, :m], w[b, j]) and (new_w[b, m:] == -1.0).all()
    keep = [p for p in range(g.kv_cache.shape[0]) if p not in free]
    assert torch.equal(g.kv_cache[keep], before[keep])


def test_evict_on_a_stream_of_its_own_fills_what_it_allocates_there(cuda_device):
    """The current stream is busy: nothing it does later may touch the results of another stream."""
    lens, budget = [900, 77], 128
    g, out_cache, out_tables = evict_inputs(lens, "bf16", budget, 31, cuda_device)
    w = 0.5 + torch.rand(2, 900, device=cuda_device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(50_000_000)  # some 25 ms
        got = mla.cache_evict(w, g.seq_lens, g.kv_cache, g.block_tables, out_cache, out_tables, budget, 4, 16,
                              stream=stream)
        torch.cuda.synchronize()
        check_evicted(g, w, budget, 4, 16, out_cache, out_tables, got)
        assert (got[2][0] >= 0.5).all()


def test_evict_reports_bad_pages_and_lengths(cuda_device):
    g, out_cache, out_tables = evict_inputs([300, 200, 100], "fp8", 128, 5, cuda_device)
    tables, to = g.block_tables.clone(), out_tables.clone()
    tables[0, 0], to[1, 1] = g.kv_cache.shape[0] + 5, -3
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    w = torch.rand(3, 300, device=cuda_device)
    lens, kept, _ = mla.cache_evict(w, g.seq_lens, g.kv_cache, tables, out_cache, to, 128, 64, 64,
                                    device_status=status)
    assert int(status) == mla.MLA_DEV_BAD_PAGE
    rows = out_cache.view(torch.uint8).view(-1, 576)[out_tables[0].long().repeat_interleave(64) * 64 +
                                                    torch.arange(128, device=cuda_device) % 64]
    assert (rows[:64] == 0).all()  # source rows that do not exist arrive as zeros
    status.zero_()
    long = torch.tensor([301, -4, 100], dtype=torch.int32, device=cuda_device)
    lens, _, _ = mla.cache_evict(w, long, g.kv_cache, g.block_tables, out_cache, out_tables, 128,
                                 device_status=status)
    assert int(status) == mla.MLA_DEV_SEQ_TOO_LONG and lens.tolist() == [128, 0, 100]


def session(g, budget, window, sinks, dtype, device):
    """The buffers of a decode step, the weights it adds and an eviction."""
    s = dict(dec=mla.MlaDecoder(g.batch, g.q_len, g.heads, g.max_seq_len, dtype, device, window=window, sinks=sinks))
    s["weights"] = torch.zeros(g.batch, g.max_seq_len, device=device)
    per = (budget + 63) // 64
    s["out_cache"] = torch.full((g.batch * per + 1, 64, 576), math.nan, device=device).to(g.kv_cache.dtype)
    s["tables"] = torch.randperm(g.batch * per + 1, generator=torch.Generator().manual_seed(1))[:g.batch * per].to(
        torch.int32).view(g.batch, per).to(device)
    s["out"] = torch.empty(g.batch, g.q_len, g.heads, 512, dtype=torch.bfloat16, device=device)
    s["lse"] = torch.empty(g.batch, g.q_len, g.heads, device=device)
    s["lens"] = torch.empty(g.batch, dtype=torch.int32, device=device)
    s["kept"] = torch.empty(g.batch, budget, dtype=torch.int32, device=device)
    s["new_weights"] = torch.zeros(g.batch, budget, device=device)
    s["after"] = mla.MlaDecoder(g.batch, g.q_len, g.heads, budget, dtype, device)
    s["out2"], s["lse2"] = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    return s


def run_session(s, g, budget, recent):
    """Attention, its weights, the eviction they decide, and attention over what stayed."""
    s["dec"](g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale, out=s["out"],
             lse=s["lse"])
    s["dec"].key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, s["lse"], s["weights"],
                         weights=s["weights"], decay=0.0, q_scale=g.q_scale, kv_scale=g.kv_scale)
    mla.cache_evict(s["weights"], g.seq_lens, g.kv_cache, g.block_tables, s["out_cache"], s["tables"], budget, 4,
                    recent, out_seq_lens=s["lens"], kept=s["kept"], out_weights=s["new_weights"])
    s["after"](g.q, s["out_cache"], s["tables"], s["lens"], g.softmax_scale, g.q_scale, g.kv_scale, out=s["out2"],
               lse=s["lse2"])


def check_session(s, g, budget, recent, window, sinks, what):
    check_attention(g, s["out"], s["lse"], window, sinks, "auto", what)
    w, tol = ref.key_weights(g, s["lse"].view(-1, g.heads), None, 0.0, g.max_seq_len, window, sinks)
    ref.close(s["weights"], w, tol, what + " weights")
    kept = ref.evict(s["weights"], g.seq_lens.tolist(), budget, 4, recent)
    assert [r[r >= 0].tolist() for r in s["kept"].cpu()] == kept
    small = type(g)(**{**g.__dict__, "kv_cache": s["out_cache"], "block_tables": s["tables"], "seq_lens": s["lens"]})
    check_attention(small, s["out2"], s["lse2"], 0, 0, "auto", what + " after")
    assert s["dec"].status() == 0 and s["after"].status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 4)])
def test_attention_weights_eviction_and_attention_again(cuda_device, dtype, window, sinks):
    budget, recent = 257, 32
    g = make_inputs_custom(3, 2, 32, dtype, [900, 257, 130], seed=31, pool=1.5).to(cuda_device)
    s = session(g, budget, window, sinks, dtype, cuda_device)
    run_session(s, g, budget, recent)
    check_session(s, g, budget, recent, window, sinks, dtype)


def test_captured_on_another_stream_and_replayed_on_new_inputs(cuda_device):
    budget, recent = 200, 32
    make = lambda seed: make_inputs_custom(3, 2, 32, "fp8", [900, 257, 130], seed=seed, pool=1.5)  # noqa: E731
    g = make(51).to(cuda_device)
    s = session(g, budget, 300, 4, "fp8", cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_session(s, g, budget, recent)
    torch.cuda.current_stream().wait_stream(side)
    check_session(s, g, budget, recent, 300, 4, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_session(s, g, budget, recent)
    for seed, lens in ((52, [900, 257, 130]), (53, [64, 899, 2])):
        new = make(seed).to(cuda_device)
        g.q.copy_(new.q)
        g.kv_cache.copy_(new.kv_cache)
        g.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.block_tables.copy_(torch.arange(3 * g.block_tables.shape[1], dtype=torch.int32).view(3, -1)
                             .clamp(max=g.kv_cache.shape[0] - 1))
        g.q_scale, g.kv_scale = g.q_scale, g.kv_scale  # captured by value
        s["weights"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_session(s, g, budget, recent, 300, 4, f"replay {seed}")
