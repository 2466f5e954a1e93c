"""Edge calls of the long-context operators on the GPU: lengths above the plan's, rows that are left out, sums of very
many rows, results packed into shared buffers. Plain 64-bit forms and bounds as in long_context_ref.py."""
import math
import time

import pytest
import torch

import long_context_ref as ref
import long_context_tight as tight
import mla_paged_decode_04_b200 as mla
from mla_paged_decode_04_b200 import _lib
from mla_paged_decode_04_b200.inputs import make_inputs_custom, make_prefill_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("planned,lens,heads,window,sinks", [
    (100, [200], 16, 4096, 4),            # two pages more than the plan's two
    (64, [65], 16, 128, 4),               # one key more
    (100, [200], 16, 200, 4),
    (64, [2000], 32, 4096, 4),
    (64, [1, 2000, 64, 700], 32, 1500, 70),
    (640, [5000, 641, 0], 128, 300, 4),   # the window bounds the pages, not the plan
])
def test_a_length_above_the_plans_is_computed_with_sinks_too(cuda_device, planned, lens, heads, window, sinks, dtype):
    """Without sinks such a length sets MLA_DEV_SEQ_TOO_LONG and is computed as far as the table goes; with sinks, whose
    plans launch only the pairs that the plan's lengths can use, it is too."""
    g = make_inputs_custom(len(lens), 1, heads, dtype, lens, seed=90, pool=1.5).to(cuda_device)
    out = torch.full((len(lens), 1, heads, 512), math.nan, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((len(lens), 1, heads), math.nan, device=cuda_device)
    for s in (0, sinks):
        dec = mla.MlaDecoder(len(lens), 1, heads, planned, dtype, cuda_device, window=window, sinks=s)
        dec(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale, out=out, lse=lse)
        assert dec.status() == mla.MLA_DEV_SEQ_TOO_LONG
        o, l, tol, ltol = ref.attention(g, window, s)
        ref.close(out.reshape(o.shape), o, tol, f"{s} sinks out")
        ref.close(lse.reshape(l.shape), l, ltol, f"{s} sinks lse")
        out.fill_(math.nan)
        lse.fill_(math.nan)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_length_above_a_prefill_plans_is_computed_with_sinks_too(cuda_device, dtype):
    g = make_prefill_inputs([37, 0, 3], [900, 10, 300], 24, dtype, seed=91).to(cuda_device)
    pre = mla.MlaPrefill(3, 37, 24, 64, dtype, cuda_device, window=800, sinks=4)
    out, lse = pre(g.q, g.cu_seqlens_q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale)
    assert pre.status() == mla.MLA_DEV_SEQ_TOO_LONG
    o, l, tol, ltol = ref.attention(g, 800, 4)
    ref.close(out.reshape(o.shape), o, tol, "out")
    ref.close(lse.reshape(l.shape), l, ltol, "lse")


# (T, H, dtype, window): every form of the tensor-core kernel, by type and rows per entry
FORMS = [(1, 16, "bf16", 0), (2, 50, "fp16", 0), (4, 32, "fp8", 0), (2, 90, "fp8", 0), (2, 100, "bf16", 0),
         (5, 128, "fp8", 0), (5, 128, "fp16", 0), (5, 128, "bf16", 150), (3, 65, "fp8", 150)]


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("T,H,dtype,window", FORMS)
def test_rows_left_out_by_their_lse_add_nothing_whatever_they_hold(cuda_device, T, H, dtype, window, kernel):
    """Padding rows of a step: lse set to -inf, q never written (NaN here), also where every row sees every key."""
    g = make_inputs_custom(2, T, H, dtype, [900, 333], seed=92, pool=1.5).to(cuda_device)
    dec = mla.MlaDecoder(2, T, H, 900, dtype, cuda_device, kernel=kernel, window=window, sinks=4 if window else 0)
    _, lse = dec(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale)
    left = torch.zeros(2, T, H, dtype=torch.bool, device=cuda_device)
    left[0, 0, 3] = left[1, T - 1, H - 1] = left[1, 0, H // 2] = True
    lse = lse.view(2, T, H).masked_fill(left, -math.inf)
    q = g.q.clone().view(torch.uint8)
    q.view(2, T, H, -1)[left] = 0xFF  # a NaN in every type

    def weights(rows):
        return dec.key_weights(rows, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse,
                               torch.zeros(2, 900, device=cuda_device), q_scale=g.q_scale, kv_scale=g.kv_scale)

    got = weights(q.view(g.q.dtype).view(g.q.shape))
    assert dec.status() == 0
    want, tol = ref.key_weights(g, lse.reshape(-1, H), None, 1.0, 900, window, 4 if window else 0)
    ref.close(got, want, tol, f"{kernel} {dtype} {T * H} rows")
    assert torch.equal(got, weights(g.q))  # the same bits as with numbers there


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("kernel", ["simt", "auto"])
def test_key_weights_reach_as_far_as_a_length_above_the_plans(cuda_device, kernel, dtype):
    """A plan for 640 keys whose splits (three of four pages) reach to 768: every key that the attention saw gets its
    weight."""
    lens = [768, 705, 640]
    g = make_inputs_custom(3, 2, 32, dtype, lens, seed=93, pool=1.5).to(cuda_device)
    dec = mla.MlaDecoder(3, 2, 32, 640, dtype, cuda_device, kernel=kernel, split_kv=3)
    _, lse = dec(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, g.q_scale, g.kv_scale)
    assert dec.status() == mla.MLA_DEV_SEQ_TOO_LONG
    got = dec.key_weights(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale, lse,
                          torch.zeros(3, 768, device=cuda_device), q_scale=g.q_scale, kv_scale=g.kv_scale)
    assert dec.status() == mla.MLA_DEV_SEQ_TOO_LONG
    want, tol = ref.key_weights(g, lse.reshape(-1, 32), None, 1.0, 768)
    ref.close(got, want, tol, f"{kernel} {dtype}")
    assert (got[0] > 0).all() and (got[1, :705] > 0).all()


@pytest.mark.parametrize("kernel", ["simt", "auto"])
def test_sums_over_very_many_rows(cuda_device, kernel):
    """Uniform attention (q = 0, so scores are exactly 0) of 1024 new tokens of 128 heads: key j of n receives the sum
    of 1 / (keys of the row) over the rows that see it, up to 131,072 nearly equal terms.

    Bound: ex2's argument is lse * log2(e) rounded once from the given fp32 lse (at most log2(4024) < 12: half a step
    2^-21, times ln 2) and ex2 is off by 2^-22: 6e-7 a term. The CUDA-core form adds in 64 bits and rounds once,
    2^-24. The tensor-core form adds up to 64 terms in a register pair, then 3 parts, 512 row groups and 2 halves in
    fp32: (64 + 3 + 512 + 2) * 2^-24 at most."""
    new, pre, H = 1024, 3000, 128
    n = new + pre
    g = make_prefill_inputs([new], [pre], H, "bf16", seed=94).to(cuda_device)
    g.q.zero_()
    lse = torch.log(torch.arange(pre + 1, n + 1, device=cuda_device).double()).float()
    dec = mla.MlaPrefill(1, new, H, n, "bf16", cuda_device, kernel=kernel)
    got = dec.key_weights(g.q, g.cu_seqlens_q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale,
                          lse[:, None].expand(new, H).contiguous(), torch.zeros(1, n, device=cuda_device))
    assert dec.status() == 0
    p = H * torch.exp(-lse.double())  # a token's rows on each key it sees
    want = torch.cat([p.sum().expand(pre + 1), p.flip(0).cumsum(0).flip(0)[1:]])
    rel = 6e-7 + (1 if kernel == "simt" else 581) * 2.0 ** -24
    ref.close(got[0], want, rel * want, kernel)


def test_key_weights_report_in_a_workspace_that_was_put_in_place_of_the_first(cuda_device):
    g = make_inputs_custom(2, 1, 32, "bf16", [300, 200], seed=6, pool=1.5).to(cuda_device)
    dec, other = (mla.MlaDecoder(2, 1, 32, 300, "bf16", cuda_device) for _ in range(2))
    dec.workspace = other.workspace
    _, lse = dec(g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale)
    tables = g.block_tables.clone()
    tables[0, 1] = -1
    dec.key_weights(g.q, g.kv_cache, tables, g.seq_lens, g.softmax_scale, lse, torch.zeros(2, 300, device=cuda_device))
    assert dec.status() == mla.MLA_DEV_BAD_PAGE


# decode (T, H, dtype, seq_lens) or ragged (new, prefix, H, dtype): each form of the kernel, groups that end inside 32
# columns, a window with sinks
TIGHT = [
    ((4, 32, "bf16", [900, 70]), 0, 0),
    ((1, 33, "fp16", [700, 129]), 0, 0),
    ((2, 100, "fp8", [600, 257]), 0, 0),                       # 200 rows of FP8
    ((2, 120, "fp16", [515, 256]), 0, 0),                      # 240 rows of 16 bits
    ((3, 115, "fp8", [700, 300]), 0, 0),                       # 345 rows of FP8: two groups
    ((5, 128, "bf16", [513, 300]), 0, 0),
    (([130, 3, 64], [250, 900, 1], 20, "fp8"), 0, 0),          # 2600 rows an entry
    (([130, 3, 64], [250, 900, 1], 20, "fp16"), 0, 0),
    (([70, 41], [600, 333], 128, "fp8"), 90, 66),              # 8960 rows
    (([70, 41], [600, 333], 128, "bf16"), 90, 66),
]


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("case", range(len(TIGHT)))
def test_key_weights_within_a_bound_that_a_lost_row_breaks(cuda_device, case, kernel):
    shape, window, sinks = TIGHT[case]
    if isinstance(shape[0], int):
        T, H, dtype, lens = shape
        g = make_inputs_custom(len(lens), T, H, dtype, lens, seed=95 + case, pool=1.5).to(cuda_device)
        dec = mla.MlaDecoder(len(lens), T, H, g.max_seq_len, dtype, cuda_device, kernel=kernel, window=window,
                             sinks=sinks)
        args = (g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale)
    else:
        new, prefix, H, dtype = shape
        g = make_prefill_inputs(new, prefix, H, dtype, seed=95 + case).to(cuda_device)
        dec = mla.MlaPrefill(len(new), max(new), H, g.max_seq_len, dtype, cuda_device, kernel=kernel, window=window,
                             sinks=sinks)
        args = (g.q, g.cu_seqlens_q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale)
    _, lse = dec(*args, g.q_scale, g.kv_scale)
    got = dec.key_weights(*args, lse, torch.zeros(g.batch, g.max_seq_len, device=cuda_device), q_scale=g.q_scale,
                          kv_scale=g.kv_scale)
    assert dec.status() == 0
    want, tol, rows = tight.key_weights(g, lse.reshape(-1, H), g.max_seq_len, window, sinks)
    ref.close(got, want, tol, f"{kernel} case {case}")
    for b, p in enumerate(rows):  # without any one of its rows an entry would be out of bounds somewhere
        assert p is None or (p > 2 * tol[b, :p.shape[1]]).any(1).all()


def test_16_bit_scores_of_few_rows_lose_less_to_cut_sums(cuda_device):
    """The tensor cores cut partial sums toward zero, at a unit of their own size. Scores of at most 64 rows go to four
    accumulators. With positive q and k (64-dim chunks of about 36, 3 + 2 + 2 + 2 of them an accumulator) the units
    met on the way add up to a quarter of one accumulator's: 13.7 against 3.6 units of 2^-24 of the score, whatever
    share of a unit an addition loses. So the mean loss has to be less than half that of 96 rows, which have one."""
    n, scale = 4096, 30 / 324
    gen = torch.Generator(device=cuda_device).manual_seed(7)
    positive = lambda *s: (0.5 + 0.5 * torch.rand(*s, generator=gen, device=cuda_device)).half()  # noqa: E731
    k, q = positive(n // 64, 64, 576), positive(1, 1, 1, 576)
    tables = torch.arange(n // 64, dtype=torch.int32, device=cuda_device)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=cuda_device)
    s = (k.view(n, 576).double() @ q.view(576).double()) * scale
    lost = []
    for heads in (1, 64, 96):
        lse = torch.full((1, 1, heads), -math.inf, device=cuda_device)
        lse[0, 0, 0] = 30.0  # one row counts
        dec = mla.MlaDecoder(1, 1, heads, n, "fp16", cuda_device)
        w = dec.key_weights(q.expand(1, 1, heads, 576).contiguous(), k, tables, lens, scale, lse,
                            torch.zeros(1, n, device=cuda_device))
        lost.append(float((s - 30.0 - w[0].double().log()).mean()))
    assert 0 < lost[0] < lost[2] / 2 and 0 < lost[1] < lost[2] / 2, lost


def test_evicted_weights_arrive_with_every_bit(cuda_device):
    """NaN among the weights: what is gathered is compared by its bits (NaN differs from itself)."""
    lens, budget, sinks, recent = [1000, 777, 3000], 200, 3, 20
    g = make_inputs_custom(3, 1, 1, "fp16", lens, seed=17, pool=1.2).to(cuda_device)
    w = torch.randn(3, 3000, generator=torch.Generator().manual_seed(1))
    w = torch.where(w > -1.2, math.nan, w).to(cuda_device)
    per = (budget + 63) // 64
    out_cache = torch.zeros(3 * per, 64, 576, dtype=torch.float16, device=cuda_device)
    out_tables = torch.arange(3 * per, dtype=torch.int32, device=cuda_device).view(3, per)
    _, kept, out_w = mla.cache_evict(w, g.seq_lens, g.kv_cache, g.block_tables, out_cache, out_tables, budget, sinks,
                                     recent)
    for b, want in enumerate(ref.evict(w, lens, budget, sinks, recent)):
        assert kept[b].tolist() == want
        assert torch.equal(out_w[b].view(torch.int32), w[b, want].view(torch.int32))
        assert torch.isnan(out_w[b]).any() and not torch.isnan(out_w[b]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("kernel", ["simt", "auto"])
def test_key_weights_and_eviction_through_the_bounds_checking_build(cuda_device, dtype, kernel, monkeypatch):
    """No check fires on valid calls, and the results are the normal build's, bit for bit."""
    long = torch.rand(2, 12000, generator=torch.Generator().manual_seed(3)).to(cuda_device)

    def run():
        res = []
        for T, H, lens, window, sinks in ((4, 32, [1000, 391, 0], 0, 0), (3, 100, [700, 65, 1], 90, 66)):
            g = make_inputs_custom(3, T, H, dtype, lens, seed=96, pool=2.0).to(cuda_device)
            dec = mla.MlaDecoder(3, T, H, 1000, dtype, cuda_device, kernel=kernel, window=window, sinks=sinks)
            args = (g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale)
            _, lse = dec(*args, g.q_scale, g.kv_scale)
            w = dec.key_weights(*args, lse, torch.zeros(3, 1000, device=cuda_device), q_scale=g.q_scale,
                                kv_scale=g.kv_scale)
            assert dec.status() == 0
            out_cache = torch.zeros(16, 64, 576, device=cuda_device).to(g.kv_cache.dtype)
            out_tables = torch.arange(15, dtype=torch.int32, device=cuda_device).view(3, 5)
            status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
            got = mla.cache_evict(w, g.seq_lens, g.kv_cache, g.block_tables, out_cache, out_tables, 300, 4, 32,
                                  device_status=status)
            assert int(status) == 0
            res += [w, out_cache.view(torch.uint8), *got]
        # a cluster an entry
        g = make_inputs_custom(2, 1, 1, dtype, [12000, 5], seed=97, pool=1.1).to(cuda_device)
        out_cache = torch.zeros(8, 64, 576, device=cuda_device).to(g.kv_cache.dtype)
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        got = mla.cache_evict(long, g.seq_lens, g.kv_cache, g.block_tables, out_cache,
                              torch.arange(8, dtype=torch.int32, device=cuda_device).view(2, 4), 200, 4, 32,
                              device_status=status)
        assert int(status) == 0
        return res + [out_cache.view(torch.uint8), *got]

    want = run()
    monkeypatch.setattr(_lib, "_lib", _lib.load_library(_lib.CHECK_LIB_PATH))
    assert mla.bounds_checked()
    for a, b in zip(run(), want):
        assert torch.equal(a, b)


# (T, H): the forms of FP8 weights: up to 128 rows, up to 256, and more
FP8_FORMS = [(4, 32), (2, 100), (3, 115)]


@pytest.mark.parametrize("T,H", FP8_FORMS)
def test_a_wait_of_key_weights_that_runs_out(cuda_device, T, H):
    """A plan in its failure-detection mode: no pair loads its first ring slot, so the MMA issuer's wait for it ends
    after its limit, every other role gives up in turn and the kernel returns with MLA_DEV_TIMEOUT. The next call on the
    same buffers is clean."""
    g = make_inputs_custom(2, T, H, "fp8", [3000, 1200], seed=98, pool=2.0).to(cuda_device)
    dec = mla.MlaDecoder(2, T, H, 3000, "fp8", cuda_device)
    args = (g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale)
    _, lse = dec(*args, g.q_scale, g.kv_scale)
    w = torch.zeros(2, 3000, device=cuda_device)
    kw = dict(q_scale=g.q_scale, kv_scale=g.kv_scale)
    want = dec.key_weights(*args, lse, w.clone(), **kw)
    torch.cuda.synchronize()
    assert dec.status() == 0
    faulty = type(dec.plan).from_buffer_copy(dec.plan)
    faulty.fault_test = 1
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    t0 = time.perf_counter()
    mla.key_weights(faulty, *args, lse, w, status, **kw)
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert int(status) == mla.MLA_DEV_TIMEOUT
    assert 0.3 < waited < 20.0, waited
    again = dec.key_weights(*args, lse, torch.zeros_like(want), **kw)
    assert dec.status() == 0 and torch.equal(again, want)


@pytest.mark.parametrize("T,H", FP8_FORMS)
def test_key_weights_past_their_rows_are_caught(cuda_device, T, H, monkeypatch):
    """The checking build with the plan's second test mode: every weight would go past its row, and is not written."""
    monkeypatch.setattr(_lib, "_lib", _lib.load_library(_lib.CHECK_LIB_PATH))
    g = make_inputs_custom(2, T, H, "fp8", [900, 333], seed=99, pool=2.0).to(cuda_device)
    dec = mla.MlaDecoder(2, T, H, 900, "fp8", cuda_device)
    args = (g.q, g.kv_cache, g.block_tables, g.seq_lens, g.softmax_scale)
    _, lse = dec(*args, g.q_scale, g.kv_scale)
    wide = torch.full((3, 900), -3.0, device=cuda_device)  # a row more than the call is given
    kw = dict(q_scale=g.q_scale, kv_scale=g.kv_scale)
    faulty = type(dec.plan).from_buffer_copy(dec.plan)
    faulty.fault_test = 2
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    mla.key_weights(faulty, *args, lse, wide[:2], status, **kw)
    assert int(status) == mla.MLA_DEV_BOUNDS and (wide == -3.0).all()
    dec.key_weights(*args, lse, wide[:2], **kw)
    assert dec.status() == 0 and (wide[0] >= 0).all() and (wide[2] == -3.0).all()


@pytest.mark.parametrize("kernel", ["simt", "auto"])
def test_pages_past_32_bit_offsets(cuda_device, kernel):
    """The same step on the last pages of a cache of 2.2e9 elements, and an eviction to the pages before them."""
    lens, pages = [1500, 700, 300], 60000
    g = make_inputs_custom(3, 4, 32, "bf16", lens, seed=101, pool=1.0).to(cuda_device)
    big = torch.empty(pages, 64, 576, dtype=torch.bfloat16, device=cuda_device)
    shift = pages - g.kv_cache.shape[0]
    big[shift:] = g.kv_cache
    tables = torch.where(g.block_tables >= 0, g.block_tables + shift, g.block_tables)
    dec = mla.MlaDecoder(3, 4, 32, 1500, "bf16", cuda_device, kernel=kernel, window=600, sinks=70)
    results = []
    for cache, table in ((g.kv_cache, g.block_tables), (big, tables)):
        out, lse = dec(g.q, cache, table, g.seq_lens, g.softmax_scale)
        w = dec.key_weights(g.q, cache, table, g.seq_lens, g.softmax_scale, lse,
                            torch.zeros(3, 1500, device=cuda_device))
        assert dec.status() == 0
        results.append((out, lse, w))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    out_tables = torch.arange(12, dtype=torch.int32, device=cuda_device).view(3, 4) + shift - 12
    _, kept, _ = mla.cache_evict(w, g.seq_lens, big, tables, big, out_tables, 256, 4, 100)
    rows = big.view(-1, 576)
    for b, want in enumerate(ref.evict(w, lens, 256, 4, 100)):
        assert kept[b, :len(want)].tolist() == want
        j, i = torch.tensor(want, device=cuda_device), torch.arange(len(want), device=cuda_device)
        to = out_tables[b].long()[i // 64] * 64 + i % 64
        assert torch.equal(rows[to], rows[tables[b].long()[j // 64] * 64 + j % 64])
