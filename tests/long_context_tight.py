"""Received key weights in 64 bits with a bound close to what the kernels round, and what losing one row would change.

The bound of long_context_ref.py adds the roundings of a dot product up as if all went one way, 1.1e-3 of a weight,
which hides a lost row among 900. Here, for a row r and a key j:
  score   each of the 577 addends of a dot product (576 products and what is there) may be cut to 24 bits of the
          largest magnitude met on the way, A = max |partial sum| + max |product|: 2^-23 A each, of either sign where
          the data is, so sqrt(577) of them, times 4
  weight  the rounded scale, the rounded lse * log2(e) and their sum: 2^-24 (2 |s| + 2 |lse| + |s - lse|); ex2 2^-22
  sum     at most 128 terms of a row group in one accumulator, then the groups and the halves: (134 + groups) 2^-24
"""
import math

import torch

from long_context_ref import entries, entry_keys, visible

STEP = 16  # dims between two looks at the partial sum


def key_weights(inp, lse, cols, window=0, sinks=0):
    """(weights [B, cols], bound, per entry the rows' probabilities [rows, n]); no old weights. lse: packed [rows, H]."""
    out = torch.zeros(len(inp.seq_lens), cols, dtype=torch.float64, device=inp.q.device)
    tol = torch.zeros_like(out)
    rows, at = [], 0
    for b, q, n in entries(inp):
        T, H = q.shape[:2]
        l = lse[at:at + T].double()
        at += T
        if n == 0 or T == 0:
            rows.append(None)
            continue
        k = entry_keys(inp.kv_cache, inp.block_tables[b], n, inp.kv_scale).view(n, -1, STEP)
        probs = torch.zeros(T, H, n, dtype=torch.float64, device=q.device)
        for t in range(T):
            qd = (q[t].double() * inp.q_scale * inp.softmax_scale).view(H, -1, STEP)
            partial = torch.einsum("hcd,ncd->hnc", qd, k).cumsum(2)
            s = partial[..., -1]
            most = partial.abs().amax(2) + qd.abs().amax((1, 2))[:, None] * k.abs().amax((1, 2))[None]
            seen = torch.zeros(n, dtype=torch.bool, device=q.device)
            seen[visible(n - T + t + 1, window, sinks)] = True
            seen = seen[None] & (l[t] > -math.inf)[:, None]
            lr = torch.where(l[t] == -math.inf, 0.0, l[t])[:, None]
            p = torch.where(seen, torch.exp(s - lr), 0.0)
            per = 4 * math.sqrt(577) * 2.0 ** -23 * most
            per = per + 2.0 ** -24 * (2 * s.abs() + 2 * lr.abs() + (s - lr).abs()) + 2.0 ** -22
            tol[b, :n] += (p * per).sum(0)
            probs[t] = p
        out[b, :n] = probs.sum((0, 1))
        tol[b, :n] += (134 + T * H / 128) * 2.0 ** -24 * out[b, :n] + 1e-37
        rows.append(probs.view(T * H, n))
    return out, tol, rows
