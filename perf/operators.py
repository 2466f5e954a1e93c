"""Long-context operators of the latent cache, measured: attention through a sliding window with attention sinks,
the attention weight each cached key received, and the eviction of the keys that received least.

`run` computes them from elementary torch operations in 32 bits (`own = False`) or through the library
(`own = True`). Layouts are the library's: a latent cache [pages, 64, 576] read through block tables, K all 576
dims and V the first 512; a query token t of an entry with n keys and T new tokens sees keys 0 .. n - T + t, of which
a window W keeps the last W and `sinks` the first few.
"""
import math

import torch

own = False

D, DV, PAGE = 576, 512, 64
SCALE = D ** -0.5
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
FP8_SCALE = 5.25 / 448.0  # |N(0, 1)| stays below 5.25 but for a few values in a million, which saturate


def listed():
    return [
        # a short chat turn of one request: what a call costs when there is hardly any work
        dict(name="window_one_request", op="window", dtype="bf16", batch=1, q_len=1, heads=16, len_lo=1500,
             len_hi=1500, new_lo=0, window=256, sinks=4),
        # speculative decoding of long agent sessions that only keep a window
        dict(name="window_agents_fp8", op="window", dtype="fp8", batch=16, q_len=4, heads=32, len_lo=81920,
             len_hi=81920, new_lo=0, window=4096, sinks=4),
        # mixed lengths, odd window and sinks, two query groups an entry
        dict(name="window_mixed_fp16", op="window", dtype="fp16", batch=32, q_len=4, heads=64, len_lo=1024,
             len_hi=65536, new_lo=0, window=2047, sinks=17),
        # many short and long requests at once, some shorter than the window or than the step
        dict(name="window_many_bf16", op="window", dtype="bf16", batch=128, q_len=2, heads=128, len_lo=1,
             len_hi=16384, new_lo=0, window=1024, sinks=64),
        # a chunk of several prompts on top of cached prefixes
        dict(name="window_prefill_fp8", op="window", dtype="fp8", batch=8, q_len=1024, heads=32, len_lo=640,
             len_hi=17408, new_lo=128, window=1024, sinks=4),
        # weights after one decode step of one request
        dict(name="weights_one_request", op="weights", dtype="bf16", batch=1, q_len=1, heads=16, len_lo=777,
             len_hi=777, new_lo=0, window=0, sinks=0, decay=1.0),
        # weights after a speculative step
        dict(name="weights_step_bf16", op="weights", dtype="bf16", batch=4, q_len=4, heads=32, len_lo=8192,
             len_hi=8192, new_lo=0, window=0, sinks=0, decay=1.0),
        # the same on the longest sessions
        dict(name="weights_agents_fp8", op="weights", dtype="fp8", batch=16, q_len=4, heads=32, len_lo=81920,
             len_hi=81920, new_lo=0, window=0, sinks=0, decay=0.9),
        # the last tokens of each prompt vote on the prompt's keys
        dict(name="weights_observe_fp16", op="weights", dtype="fp16", batch=4, q_len=32, heads=64, len_lo=4097,
             len_hi=32768, new_lo=16, window=0, sinks=0, decay=0.0),
        # one request that has just outgrown its budget
        dict(name="evict_one_request", op="evict", dtype="bf16", batch=1, len_lo=1100, len_hi=1100, budget=1024,
             sinks=4, recent=128),
        # mixed lengths, some below the budget
        dict(name="evict_mixed_bf16", op="evict", dtype="bf16", batch=64, len_lo=1000, len_hi=16384, budget=2000,
             sinks=7, recent=333),
        # the longest sessions cut to a tenth
        dict(name="evict_agents_fp8", op="evict", dtype="fp8", batch=16, len_lo=81920, len_hi=81920, budget=8192,
             sinks=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "weights", "evict"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp8"]))
    if op == "evict":
        hi = _log(rng, 300, 65536)
        budget = _log(rng, 64, max(64, min(8192, hi)))
        c.update(batch=_log(rng, 1, min(64, max(1, (1 << 20) // hi))), len_lo=rng.randint(0, hi), len_hi=hi,
                 budget=budget, sinks=rng.randint(0, min(64, budget // 4)), recent=rng.randint(0, budget // 2))
        return c
    prefill = rng.random() < 0.35
    heads = rng.choice([1, 5, 8, 16, 32, 33, 64, 96, 128])
    if op == "window":
        q_len = _log(rng, 2, 512) if prefill else rng.randint(1, 4)
        hi = _log(rng, 256, 65536)
        batch = _log(rng, 1, max(1, min(8 if prefill else 64, (1 << 19) // hi, (1 << 16) // (q_len * heads) + 1)))
        window = _log(rng, 16, 8192)
        sinks = rng.choice([0, 1, 4, rng.randint(2, 200)])
    else:
        q_len = _log(rng, 2, 64) if prefill else rng.randint(1, 4)
        hi = _log(rng, 256, 65536)
        batch = _log(rng, 1, max(1, min(16, (1 << 19) // hi, (1 << 27) // (q_len * heads * hi) + 1)))
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        sinks = rng.randint(0, 64) if window else 0
        c.update(decay=rng.choice([0.0, 0.5, 1.0]))
    c.update(batch=batch, q_len=q_len, heads=heads, len_lo=rng.randint(0, hi), len_hi=hi,
             new_lo=rng.randint(1, q_len) if prefill else 0, window=window, sinks=sinks)
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _lengths(case):
    """Per entry: keys in the cache, and new tokens among them (q_len each where `new_lo` is 0)."""
    n = _spread(case["len_lo"], case["len_hi"], case["batch"])
    if case["op"] == "evict":
        return n, None
    if not case["new_lo"]:
        return n, [case["q_len"]] * case["batch"]
    return n, [min(a, b) for a, b in zip(_spread(case["new_lo"], case["q_len"], case["batch"]), n)]


def _cache(case, tables, gen, pages):
    x = torch.randn(pages * PAGE, D, generator=gen, device="cuda")
    if case["dtype"] == "fp8":
        x = (x / FP8_SCALE).clamp_(-448.0, 448.0)
    return x.to(TORCH[case["dtype"]]).view(pages, PAGE, D)


def _tables(lens, gen, pages_of=None):
    """A block table of distinct pages out of a shuffled pool a quarter larger than needed; -1 behind an entry."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    width = max(1, max(need))
    total = sum(need)
    pool = total + total // 4 + 1
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    cnt = torch.tensor(need, device="cuda")
    first = torch.cumsum(cnt, 0) - cnt
    at = first[:, None] + col[None]
    return torch.where(col[None] < cnt[:, None], perm[at.clamp(max=pool - 1)], -1).to(torch.int32), pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, new = _lengths(case)
    order = torch.randperm(len(lens), generator=gen, device="cuda").tolist()
    lens = [lens[i] for i in order]
    B = len(lens)
    s = dict(case=case, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len=max(1, max(lens)))
    s["tables"], pages = _tables(lens, gen)
    s["cache"] = _cache(case, s["tables"], gen, pages)
    fp8 = case["dtype"] == "fp8"
    s["q_scale"] = s["kv_scale"] = FP8_SCALE if fp8 else 1.0
    if case["op"] == "evict":
        # what each key received is spread over orders of magnitude, and some keys received nothing
        w = torch.exp(2.0 * torch.randn(B, s["max_len"], generator=gen, device="cuda"))
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.02, 0.0, w)
        s["out_tables"], out_pages = _tables([case["budget"]] * B, gen)
        s["out_cache"] = torch.zeros(out_pages, PAGE, D, dtype=TORCH[case["dtype"]], device="cuda")
        s["kept"] = torch.empty(B, case["budget"], dtype=torch.int32, device="cuda")
        s["out_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["out_weights"] = torch.zeros(B, case["budget"], device="cuda")
        return s
    new = [new[i] for i in order]
    T, H = case["q_len"], case["heads"]
    s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    s["cu"] = torch.nn.functional.pad(torch.cumsum(s["new"], 0), (1, 0)).to(torch.int32)
    s["total"] = sum(new)
    q = torch.randn(s["total"], H, D, generator=gen, device="cuda")
    if fp8:
        q = (q / FP8_SCALE).clamp_(-448.0, 448.0)
    q = q.to(TORCH[case["dtype"]])
    s["ragged"] = bool(case["new_lo"])
    s["q"] = q if s["ragged"] else q.view(B, T, H, D)
    lead = (s["total"], H) if s["ragged"] else (B, T, H)
    if case["op"] == "window":
        s["out"] = torch.zeros(*lead, DV, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(lead, device="cuda")
    else:
        # the attention's own log-sum-exp comes with its output, entry by entry here
        s["lse"] = torch.full((s["total"], H), -math.inf, device="cuda")
        at = 0
        for b in range(B):
            if new[b] and lens[b]:
                k = _rows(s["cache"], s["tables"][b:b + 1], torch.arange(lens[b], device="cuda")[None])[0]
                sc = _flat(s["q"])[at:at + new[b]].float().reshape(-1, D) @ k.float().T
                sc *= SCALE * s["q_scale"] * s["kv_scale"]
                j = torch.arange(lens[b], device="cuda")[None]
                last = (lens[b] - new[b] + torch.arange(new[b], device="cuda")).repeat_interleave(H)[:, None]
                sc.masked_fill_(~_sees(j, last, case), -math.inf)
                s["lse"][at:at + new[b]] = torch.logsumexp(sc, 1).view(new[b], H)
            at += new[b]
        s["lse"] = s["lse"].view(lead)
        s["before"] = torch.rand(B, s["max_len"], generator=gen, device="cuda")
        s["after"] = torch.zeros(B, s["max_len"], device="cuda")
    if own:
        import mla_paged_decode_04_b200 as mla

        kind = mla.MlaPrefill if s["ragged"] else mla.MlaDecoder
        s["attn"] = kind(B, T, H, s["max_len"], case["dtype"], "cuda", window=case["window"], sinks=case["sinks"])
    return s


def _flat(q):
    return q.reshape(-1, q.shape[-2], q.shape[-1])


def _rows(cache, tables, pos):
    """The cache's rows of each entry at positions `pos` [B, n]; any row where the position has no page."""
    page = torch.gather(tables, 1, (pos // PAGE).clamp(0, tables.shape[1] - 1)).clamp(min=0)
    at = page.long() * PAGE + pos.clamp(min=0) % PAGE
    return cache.view(-1, D)[at] if cache.dtype != torch.float8_e4m3fn else \
        cache.view(torch.uint8).view(-1, D)[at].view(torch.float8_e4m3fn)


def _sees(j, last, case):
    """Which keys j a token whose newest key is `last` attends to."""
    seen = (j >= 0) & (j <= last)
    return seen & ((j > last - case["window"]) | (j < case["sinks"])) if case["window"] else seen


def _padded(s):
    """The query rows as [B, T, H, 576] in fp32, each token's newest key [B, T] (-1: no token), and where the packed
    tokens sit in it."""
    case = s["case"]
    B, T, H = case["batch"], case["q_len"], case["heads"]
    t = torch.arange(T, device="cuda")[None]
    last = torch.where(t < s["new"][:, None], s["seq_lens"][:, None] - s["new"][:, None] + t, -1)
    if not s["ragged"]:
        return s["q"].float() * s["q_scale"], last, None
    ent = torch.repeat_interleave(torch.arange(B, device="cuda"), s["new"].long(), output_size=s["total"])
    at = ent * T + torch.arange(s["total"], device="cuda") - s["cu"][:-1].long()[ent]
    q = torch.zeros(B * T, H, D, device="cuda")
    q[at] = s["q"].float() * s["q_scale"]
    return q.view(B, T, H, D), last, at


def _window_plain(s):
    case = s["case"]
    B, T, H = case["batch"], case["q_len"], case["heads"]
    q, last, at = _padded(s)
    first = (s["seq_lens"] - s["new"] + 1 - case["window"])[:, None]  # where the first token's window begins
    span = torch.arange(min(case["window"] + T - 1, s["max_len"] + T), device="cuda")[None]
    near = first.clamp(min=0) + span
    near = torch.where(near >= case["sinks"], near, -1)
    pos = torch.cat([torch.arange(case["sinks"], device="cuda")[None].expand(B, -1), near], 1)
    k = _rows(s["cache"], s["tables"], pos).float() * s["kv_scale"]
    sc = torch.matmul(q.view(B, T * H, D), k.transpose(1, 2)).view(B, T, H, -1) * SCALE
    seen = _sees(pos[:, None], last[:, :, None], case)
    sc.masked_fill_(~seen[:, :, None], -math.inf)
    m = sc.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m)
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(B, T * H, -1), k[..., :DV]).view(B, T, H, DV)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total)).squeeze(3)
    if at is not None:
        o, lse = o.view(B * T, H, DV)[at], lse.view(B * T, H)[at]
    s["out"].copy_(o)
    s["lse"].copy_(lse)
    return s["out"], s["lse"]


def _weights_plain(s):
    case = s["case"]
    B, T, H = case["batch"], case["q_len"], case["heads"]
    q, last, at = _padded(s)
    lse = s["lse"]
    if at is not None:
        lse = torch.full((B * T, H), -math.inf, device="cuda")
        lse[at] = s["lse"]
    pos = torch.arange(s["max_len"], device="cuda")[None].expand(B, -1)
    k = _rows(s["cache"], s["tables"], pos).float() * s["kv_scale"]
    sc = torch.matmul(q.view(B, T * H, D), k.transpose(1, 2)).view(B, T, H, -1) * SCALE
    sc -= lse.view(B, T, H, 1)
    seen = _sees(pos[:, None], last[:, :, None], case)
    got = torch.exp(sc.masked_fill_(~seen[:, :, None], -math.inf)).view(B, T * H, -1).sum(1)
    if case["decay"]:
        got = got + case["decay"] * s["before"]
    s["after"].copy_(torch.where(pos < s["seq_lens"][:, None], got, s["after"]))
    return s["after"]


def _evict_plain(s):
    case = s["case"]
    B, budget = case["batch"], case["budget"]
    n = s["seq_lens"][:, None].long()
    j = torch.arange(s["max_len"], device="cuda")[None]
    safe = (j < case["sinks"]) | (j >= n - case["recent"])
    w = torch.where(j < n, torch.where(safe, math.inf, s["weights"]), -math.inf)
    best = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :budget]  # ties: the lowest index first
    best = torch.nn.functional.pad(best, (0, budget - best.shape[1]), value=1 << 40)
    count = n.clamp(max=budget)
    i = torch.arange(budget, device="cuda")[None]
    kept = torch.sort(torch.where(i < count, best, 1 << 40), dim=1).values
    kept = torch.where(i < count, kept, -1)
    raw = torch.uint8 if case["dtype"] == "fp8" else TORCH[case["dtype"]]
    out = s["out_cache"].view(raw).view(-1, D)
    to = torch.gather(s["out_tables"], 1, (i // PAGE).expand(B, -1)).long() * PAGE + i % PAGE
    rows = _rows(s["cache"], s["tables"], kept).view(raw)
    out[to] = torch.where((i < count)[..., None], rows, out[to])
    s["kept"].copy_(kept)
    s["out_lens"].copy_(count[:, 0])
    s["out_weights"].copy_(torch.where(i < count, torch.gather(s["weights"], 1, kept.clamp(min=0)), s["out_weights"]))
    return s["out_cache"], s["kept"], s["out_lens"], s["out_weights"]


def run(s):
    case = s["case"]
    if not own:
        return {"window": _window_plain, "weights": _weights_plain, "evict": _evict_plain}[case["op"]](s)
    if case["op"] == "evict":
        import mla_paged_decode_04_b200 as mla

        mla.cache_evict(s["weights"], s["seq_lens"], s["cache"], s["tables"], s["out_cache"], s["out_tables"],
                        case["budget"], sinks=case["sinks"], recent=case["recent"], out_seq_lens=s["out_lens"],
                        kept=s["kept"], out_weights=s["out_weights"])
        return s["out_cache"], s["kept"], s["out_lens"], s["out_weights"]
    q = (s["q"], s["cu"]) if s["ragged"] else (s["q"],)
    if case["op"] == "window":
        return s["attn"](*q, s["cache"], s["tables"], s["seq_lens"], SCALE, s["q_scale"], s["kv_scale"],
                         out=s["out"], lse=s["lse"])
    return s["attn"].key_weights(*q, s["cache"], s["tables"], s["seq_lens"], SCALE, s["lse"], s["after"],
                                 weights=s["before"] if case["decay"] else None, decay=case["decay"],
                                 q_scale=s["q_scale"], kv_scale=s["kv_scale"])


def _seen_counts(case):
    """(keys read, (row, key) pairs) that a case cannot do without."""
    lens, new = _lengths(case)
    keys = pairs = 0
    for n, t in zip(lens, new):
        w = case["window"] or n
        lo, sinks = max(0, n - t + 1 - w), case["sinks"] if case["window"] else 0
        if n and t:
            keys += max(0, n - lo) + min(lo, sinks)
        for last in range(max(0, n - t), n):
            at = max(0, last + 1 - w)
            pairs += last + 1 - at + min(at, sinks)
    return keys, pairs * case["heads"]


def work(case):
    size = 1 if case["dtype"] == "fp8" else 2
    lens, new = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * D * size + 8), "flops": sum(lens)}
    keys, pairs = _seen_counts(case)
    rows = sum(new) * case["heads"]
    if case["op"] == "window":
        return {"bytes": keys * D * size + rows * (D * size + 2 * DV + 4), "flops": 2 * pairs * (D + DV)}
    moved = sum(lens) * (8 if case["decay"] else 4)
    return {"bytes": keys * D * size + rows * (D * size + 4) + moved, "flops": 2 * pairs * D}


def exact(case, seed):
    """The definition in 64 bits, entry by entry and, for attention, a few tokens at a time."""
    s = prepare(case, seed)
    lens = s["seq_lens"].tolist()
    real = lambda rows, scale: rows.to(torch.float64) * scale  # noqa: E731

    def entry(b, n):
        p = torch.arange(n, device="cuda")
        slots = s["tables"][b].long()[p // PAGE] * PAGE + p % PAGE
        return s["cache"].view(torch.uint8).view(-1, D * s["cache"].element_size())[slots].view(s["cache"].dtype)

    if case["op"] == "evict":
        pool = s["out_cache"].to(torch.float64).view(-1, D)
        weights = s["out_weights"].to(torch.float64)
        for b, n in enumerate(lens):
            if n <= case["budget"]:
                keep = torch.arange(n, device="cuda")
            else:
                mid = torch.arange(case["sinks"], n - case["recent"], device="cuda")
                w = s["weights"][b, mid].to(torch.float64)
                many = case["budget"] - case["sinks"] - case["recent"]
                keep = torch.arange(0, device="cuda")
                if many:
                    least = torch.topk(w, many).values[-1]  # the smallest weight that stays
                    over, equal = mid[w > least], mid[w == least]
                    keep = torch.cat([over, equal[:many - len(over)]])
                ends = [torch.arange(case["sinks"], device="cuda"), torch.arange(n - case["recent"], n, device="cuda")]
                keep = torch.cat([ends[0], keep, ends[1]]).sort().values
            i = torch.arange(len(keep), device="cuda")
            pool[s["out_tables"][b].long()[i // PAGE] * PAGE + i % PAGE] = entry(b, n)[keep].to(torch.float64)
            weights[b, :len(keep)] = s["weights"][b, keep].to(torch.float64)
        return pool.view(s["out_cache"].shape), None, None, weights
    new, H = s["new"].tolist(), case["heads"]
    q = real(_flat(s["q"]), s["q_scale"])
    given = s["lse"].reshape(-1, H).to(torch.float64)
    out = torch.zeros(s["total"], H, DV, dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], H), -math.inf, dtype=torch.float64, device="cuda")
    after = s["after"].to(torch.float64) if case["op"] == "weights" else None
    at = 0
    for b, (n, t) in enumerate(zip(lens, new)):
        k = real(entry(b, n), s["kv_scale"])
        got = torch.zeros(n, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 28) // max(1, H * n))
        for t0 in range(0, t, step):
            for_ = range(t0, min(t, t0 + step))
            rows = slice(at + t0, at + for_.stop)
            z = torch.einsum("thd,nd->thn", q[rows], k) * SCALE
            hidden = torch.ones(len(for_), n, dtype=torch.bool, device="cuda")
            for i, tok in enumerate(for_):
                end = n - t + tok + 1
                if end > 0:
                    lo = max(0, end - case["window"]) if case["window"] else 0
                    hidden[i, lo:end] = False
                    if case["window"]:
                        hidden[i, :min(case["sinks"], end)] = False
            z.masked_fill_(hidden[:, None], -math.inf)
            if n and after is None:
                lse[rows] = torch.logsumexp(z, 2)
                p = torch.exp(z - torch.where(lse[rows] == -math.inf, 0.0, lse[rows])[..., None])
                out[rows] = torch.einsum("thn,nd->thd", p, k[:, :DV])
            elif n:
                base = given[rows][..., None]
                got += torch.exp(z - torch.where(base == -math.inf, 0.0, base)).sum((0, 1))
        if after is not None:
            after[b, :n] = got + (case["decay"] * s["before"][b, :n].to(torch.float64) if case["decay"] else 0.0)
        at += t
    if after is not None:
        return after
    return out.view(s["out"].shape), lse.view(s["lse"].shape)
