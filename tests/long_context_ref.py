"""Plain 64-bit forms of the long-context operators (windowed attention with sinks, received weights, eviction) and
the error bounds the GPU results are held to, from the roundings each path makes.

Bounds, for a row with probabilities p (sum 1) over its visible keys:
  score    products of 8- and 16-bit values are exact in fp32 and a dot product of 576 of them sums in fp32:
           |ds| <= 2 * 577 * 2^-24 * scale * sum_d |q_d k_d| (twice u per addition: tensor cores may truncate)
  weight   each probability is off by |ds|, by the rounding of lse * log2(e) and of the scaled score (2^-22 of their
           size), by ex2 (2^-22), and the sum over R rows in fp32 by R * 2^-24
  output   as the probabilities, with P rounded to its 16-bit type (half a step, eps / 2) or to two E4M3 terms
           (2^-4 * 2^-4, and below E4M3's normal range 2^-10 absolute where the row's largest P is at least 2^4),
           and the result rounded to BF16 (2^-8); every probability multiplies one |v|
"""
import math

import numpy as np
import torch

D, DV, PAGE = 576, 512, 64
U32 = 2.0 ** -24
P_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp8": 2.0 ** -8}


def visible(n, window, sinks):
    """Keys a row with n of them attends to, ascending."""
    if n <= 0:
        return []
    lo = max(0, n - window) if window else 0
    first = range(min(sinks, lo)) if window else range(0)
    return list(first) + list(range(lo, n))


def entry_keys(cache, table, n, scale):
    j = torch.arange(n, device=cache.device)
    at = table.long().to(cache.device)[j // PAGE] * PAGE + j % PAGE
    raw = cache.view(torch.uint8).reshape(-1, D * cache.element_size())[at]
    return raw.view(cache.dtype).double() * scale


def entries(inp):
    """(entry, its query rows [T, H, 576] as they are, keys n) of a decode or ragged input."""
    lens = inp.seq_lens.tolist()
    if hasattr(inp, "cu_seqlens_q"):
        cu = inp.cu_seqlens_q.tolist()
        return [(b, inp.q[cu[b]:cu[b + 1]], n) for b, n in enumerate(lens)]
    return [(b, inp.q[b], n) for b, n in enumerate(lens)]


def scores(inp, b, q, n, window, sinks):
    """(scores [T, H, n] with -inf where hidden, their error bound, keys [n, 576]) in 64 bits."""
    k = entry_keys(inp.kv_cache, inp.block_tables[b], n, inp.kv_scale)
    qd = q.double() * inp.q_scale
    s = torch.einsum("thd,nd->thn", qd, k) * inp.softmax_scale
    size = torch.einsum("thd,nd->thn", qd.abs(), k.abs()) * inp.softmax_scale
    hidden = torch.ones(q.shape[0], 1, n, dtype=torch.bool, device=q.device)
    for t in range(q.shape[0]):
        hidden[t, 0, visible(n - q.shape[0] + t + 1, window, sinks)] = False
    ds = 2 * 577 * U32 * size + 4 * U32 * s.abs()
    return s.masked_fill(hidden, -math.inf), ds.masked_fill(hidden, 0.0), k


def attention(inp, window=0, sinks=0, p_step=None):
    """(out [rows, H, 512], lse [rows, H], bound of out, bound of lse), rows packed over the entries."""
    step = P_STEP[inp.dtype] if p_step is None else p_step
    outs, lses, tols, ltols = [], [], [], []
    for b, q, n in entries(inp):
        T, H = q.shape[:2]
        if T == 0:
            continue
        if n == 0:
            outs.append(torch.zeros(T, H, DV).double().to(q.device))
            lses.append(torch.full((T, H), -math.inf).double().to(q.device))
            tols.append(torch.zeros_like(outs[-1]))
            ltols.append(torch.zeros_like(lses[-1]))
            continue
        s, ds, k = scores(inp, b, q, n, window, sinks)
        lse = torch.logsumexp(s, 2)
        p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        v = k[:, :DV]
        o = torch.einsum("thn,nd->thd", p, v)
        worst = ds.amax(2)
        l_tol = worst + 2.0 ** -20 + n * U32 + 2.0 ** -22 * lse.nan_to_num(neginf=0.0).abs()
        spread = torch.einsum("thn,nd->thd", p, v.abs())
        tol = 2.0 ** -8 * o.abs() + (step + 2 * worst + 2.0 ** -16)[..., None] * spread
        if inp.dtype == "fp8" and step:
            seen = (s > -math.inf).double()
            tol = tol + 2.0 ** -14 * p.amax(2)[..., None] * torch.einsum("thn,nd->thd", seen, v.abs())
        outs.append(o)
        lses.append(lse)
        tols.append(tol)
        ltols.append(l_tol)
    return torch.cat(outs), torch.cat(lses), torch.cat(tols), torch.cat(ltols)


def key_weights(inp, lse, before, decay, cols, window=0, sinks=0):
    """(weights [B, cols], bound): columns from an entry's length on are 0 with bound 0. lse: packed [rows, H]."""
    B = len(inp.seq_lens)
    out = torch.zeros(B, cols, dtype=torch.float64, device=inp.q.device)
    tol = torch.zeros_like(out)
    at = 0
    for b, q, n in entries(inp):
        T, H = q.shape[:2]
        rows = lse[at:at + T].double()
        at += T
        if n == 0:
            continue
        got, err = torch.zeros(n, device=q.device).double(), torch.zeros(n, device=q.device).double()
        if T:
            s, ds, _ = scores(inp, b, q, n, window, sinks)
            empty = rows == -math.inf
            p = torch.exp(s - torch.where(empty, 0.0, rows)[..., None])
            p = torch.where(empty[..., None], 0.0, p)
            got = p.sum((0, 1))
            per = ds + 2.0 ** -21 + 2.0 ** -22 * (torch.where(empty, 0.0, rows)[..., None].abs() + s.nan_to_num(
                neginf=0.0).abs()) + T * H * U32
            err = (p * per).sum((0, 1))
        if decay and before is not None:
            got = got + decay * before[b, :n].double()
        out[b, :n] = got
        tol[b, :n] = err + 4 * U32 * got.abs() + 1e-37
    return out, tol


def evict(weights, seq_lens, budget, sinks, recent):
    """[the positions that stay, ascending] per entry, by sorting (NaN lowest, ties to the lower position)."""
    kept = []
    for b, n in enumerate(seq_lens):
        n = max(0, min(int(n), weights.shape[1]))
        if n <= budget:
            kept.append(list(range(n)))
            continue
        mid = list(range(sinks, n - recent))
        w = weights[b].double().cpu().tolist()
        order = sorted(mid, key=lambda j: (math.isnan(w[j]), -w[j] if not math.isnan(w[j]) else 0.0, j))
        best = order[:budget - sinks - recent]
        kept.append(list(range(sinks)) + sorted(best) + list(range(n - recent, n)))
    return kept


def close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst "
                           f"{float(((got - want).abs() - tol)[bad].max()):.3e} over at "
                           f"{np.unravel_index(int((((got - want).abs() - tol).nan_to_num(nan=1e9)).argmax()), got.shape)}")
