"""Edge calls of the long-context operators on the GPU: lengths above the plan's, rows that are left out, sums of very
many rows, results packed into shared buffers. Plain 64-bit forms and bounds as in long_context_ref.py."""
import math

import pytest
import torch

import long_context_ref as ref
import mla_paged_decode_04_b200 as mla
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
