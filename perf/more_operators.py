"""The long-cache operators as they are measured: cases, inputs, plain forms and the
framework's calls.

    score    kv_bounds, then block_scores: lower and upper bounds of every channel of a
             page's keys, brought up to date for the newest tokens, and the largest score
             that a key of each page can have with a query
    select   block_select: the pages that each query reads, by those scores
    attn     attn_blocks: attention over the selected pages of a paged cache
    weights  kv_weights: the attention weight that every cached token received
    evict    kv_evict: the cache cut to a budget, tokens of the greatest weight kept

Where `own` is false, run() computes an operator from elementary torch operations in 32
bits; where it is true, it calls the framework. exact() is the definition in 64 bits,
written apart from both.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The newest token of 32 long conversations against the bounds of all their pages.
        dict(name="score decode", op="score", B=32, Hq=32, Hkv=8, d=128, Nq=1, page=64, lo=2048, hi=32768,
             ragged=False, shape=1),
        # A chunk of three long prompts, grouped keys.
        dict(name="score chunk", op="score", B=3, Hq=32, Hkv=8, d=128, Nq=512, page=64, lo=8192, hi=32768,
             ragged=True, shape=2),
        # One row for each conversation and key head: 32 pages of up to 512.
        dict(name="select decode", op="select", B=32, Hkv=8, Nq=1, page=64, lo=2048, hi=32768, ragged=False, n=32,
             first=1, last=2, shape=3),
        # A row for each token of a chunk, small pages, odd counts.
        dict(name="select chunk", op="select", B=3, Hkv=5, Nq=509, page=32, lo=4096, hi=32000, ragged=True, n=24,
             first=1, last=2, shape=4),
        # The smallest call of a chat server: four conversations, small pages, some
        # shorter than what is selected. Latency is all that counts.
        dict(name="blocks few", op="attn", B=4, Hq=16, Hkv=4, d=64, Nq=1, page=16, lo=1, hi=700, ragged=False, n=16,
             first=1, last=2, shape=5),
        # An ordinary decoding step: 2048 of up to 32768 tokens for each key head.
        dict(name="blocks decode", op="attn", B=32, Hq=32, Hkv=8, d=128, Nq=1, page=64, lo=2048, hi=32768,
             ragged=False, n=32, first=1, last=2, shape=6),
        # Checking drafted tokens: seven heads a key head, small heads, ragged counts.
        dict(name="blocks verify", op="attn", B=7, Hq=21, Hkv=3, d=32, Nq=5, page=32, lo=5, hi=9000, ragged=True, n=24,
             first=1, last=2, shape=7),
        # A chunk of two long prompts, every token with pages of its own.
        dict(name="blocks chunk", op="attn", B=2, Hq=32, Hkv=8, d=128, Nq=512, page=64, lo=4096, hi=16384, ragged=True,
             n=32, first=1, last=4, shape=8),
        # A decoding step adds its weights to those of the tokens before.
        dict(name="weights decode", op="weights", B=32, Hq=32, Hkv=8, d=128, Nq=1, page=64, lo=256, hi=4224,
             ragged=False, decay=1.0, shape=9),
        # The weights that the last tokens of three prompts give to all before them.
        dict(name="weights chunk", op="weights", B=3, Hq=15, Hkv=5, d=64, Nq=333, page=32, lo=2000, hi=12000,
             ragged=True, decay=0.0, shape=10),
        # Conversations a little over their budget, cut back to it.
        dict(name="evict step", op="evict", B=16, Hkv=5, d=64, page=16, lo=900, hi=1290, budget=1024, first=4, last=64,
             shape=11),
        # Long prompts cut to an eighth, into fresh pages.
        dict(name="evict prompt", op="evict", B=6, Hkv=8, d=128, page=64, lo=16384, hi=32768, budget=4096, first=16,
             last=256, shape=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["score", "select", "attn", "attn", "weights", "evict"])
    c = dict(op=op, B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 3, 4, 5, 8, 16]), page=rng.choice([16, 32, 64, 128]),
             shape=rng.randrange(1 << 20))
    if op != "select":
        c["d"] = rng.choice([32, 64, 128])
    if op == "evict":
        c["budget"] = _log(rng, 16, 8192)
        c["hi"] = _log(rng, c["budget"] // 2 + 1, 32768)
        c["lo"] = rng.randint(1, c["hi"])
        c["first"], c["last"] = rng.randint(0, c["budget"] // 4), rng.randint(0, c["budget"] // 2)
        return c
    c["Nq"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 512)])
    c["hi"] = _log(rng, max(c["Nq"], 16), 65536)
    c["lo"] = rng.choice([c["Nq"], max(c["Nq"], c["hi"] // 2), c["hi"]])
    c["ragged"] = c["Nq"] > 1 and rng.random() < 0.5
    if op != "select":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op in ("select", "attn"):
        c["n"] = rng.choice([4, 8, 16, 24, 32, 64])
        c["first"], c["last"] = rng.choice([0, 1, 2]), rng.choice([1, 2])
    if op == "weights":
        c["decay"] = rng.choice([0.0, 1.0, 0.9])
    return c


def draw(rng):
    """One more case, no dearer than the largest listed one of its operator."""
    while True:
        case = _draw(rng)
        top = [work(c) for c in listed() if c["op"] == case["op"]]
        w = work(case)
        tokens = sum(-(-n // case["page"]) * case["page"] for n in _lengths(case)[0])
        if tokens * case["Hkv"] * case.get("d", 0) > 1 << 29:
            continue  # a cache of this size is made many times over
        if case["op"] == "attn" and case["B"] * case["Hkv"] * case["Nq"] * case["n"] * case["page"] * case["d"] > 1 << 31:
            continue  # what the plain form gathers
        if case["op"] == "weights" and case["B"] * case["Hq"] * case["Nq"] * case["hi"] > 1 << 29:
            continue  # the plain form's scores
        if all(w[m] <= max(t[m] for t in top) for m in ("bytes", "flops")):
            return case


def _lengths(case):
    """Tokens of each sequence, spread over [lo, hi], and how many of its Nq queries are
    real. From the case alone."""
    r = random.Random(case["shape"])
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + int(round((hi - lo) * r.random() ** 1.5)) for _ in range(B)]
    lens[r.randrange(B)] = hi
    n = case.get("Nq", 1)
    new = [r.randint(1, n) if case.get("ragged") else n for _ in range(B)]
    return [max(a, b) for a, b in zip(lens, new)], new


def _width(case):
    """Entries of a sequence in the block table."""
    return max(-(-n // case["page"]) for n in _lengths(case)[0])


def work(case):
    lens, new = _lengths(case)
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    d, Nq = case.get("d", 0), case.get("Nq", 1)
    pages = [-(-n // page) for n in lens]
    W = max(pages)
    if case["op"] == "score":
        Hq = case["Hq"]
        fresh = sum(p - (n - m) // page for p, n, m in zip(pages, lens, new))
        read = 2 * Hkv * d * page * fresh + 2 * 2 * Hkv * d * sum(pages) + 2 * B * Hq * Nq * d
        return dict(bytes=read + 2 * 2 * Hkv * d * fresh + 4 * B * Hkv * Nq * W + 4 * sum(pages),
                    flops=4 * d * Hq * sum(p * m for p, m in zip(pages, new)))
    if case["op"] == "select":
        return dict(bytes=4 * Hkv * sum(p * m for p, m in zip(pages, new)) + 4 * B * Hkv * Nq * case["n"],
                    flops=2 * Hkv * sum(p * m for p, m in zip(pages, new)))
    if case["op"] == "attn":
        Hq, n = case["Hq"], case["n"]
        seen = sum(min(n * page, x) * m for x, m in zip(lens, new))       # keys, over the queries
        kept = sum(min(p, n * m) * page for p, m in zip(pages, new))      # slots that have to be read
        return dict(bytes=2 * 2 * Hkv * d * kept + 2 * 2 * B * Hq * Nq * d + 4 * B * Hq * Nq + 4 * B * Hkv * Nq * n,
                    flops=4 * d * Hq * seen)
    if case["op"] == "weights":
        Hq = case["Hq"]
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
        return dict(bytes=2 * Hkv * d * sum(lens) + (8 if case["decay"] else 4) * Hkv * sum(lens) + 2 * B * Hq * Nq * d
                    + 4 * B * Hq * Nq + 4 * sum(pages), flops=2 * d * Hq * pairs)
    kept = sum(min(n, case["budget"]) for n in lens)
    return dict(bytes=Hkv * (4 * sum(lens) + kept * (2 * 2 * 2 * d + 4) + 4 * B * case["budget"]) + 4 * sum(pages),
                flops=Hkv * sum(lens))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFFFFFF)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(counts, seed):
    """Tables over shuffled pages, one list of page counts for each; unused entries -1."""
    total = sum(sum(c) for c in counts)
    order = list(range(total))
    random.Random(seed).shuffle(order)
    out, at = [], 0
    for need in counts:
        width, rows = max(need), []
        for n in need:
            rows.append(order[at:at + n] + [-1] * (width - n))
            at += n
        out.append(_int(rows))
    return total, out


def _keys(g, case, pages, u):
    """Cached keys: a direction of each key head, and one that every page has of its own."""
    Hkv, d = case["Hkv"], case["d"]
    k = _randn(g, pages, Hkv, case["page"], d).bfloat16()
    k += (0.5 * u[:, None] + 0.7 * _randn(g, pages, Hkv, 1, d)).bfloat16()
    return k


def _queries(g, case, u):
    B, Hq, Hkv, Nq, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "d"))
    q = _randn(g, B, Hkv, Hq // Hkv, Nq, d) + 0.5 * u[:, None, None]
    return q.reshape(B, Hq, Nq, d).bfloat16()


def _visible(case, lens, new, n):
    """Pages that each query sees, [B, 1, Nq, 1] of `n`; none for a padded one."""
    i = torch.arange(case["Nq"], device="cuda")
    last = lens.long()[:, None] - new.long()[:, None] + i
    return torch.where(i < new[:, None], last // case["page"] + 1, 0).clamp(0, n)[:, None, :, None]


def _page_scores(g, case, lens, new, W):
    """Scores as trained heads give them: neighbouring tokens prefer much the same pages."""
    B, Hkv, Nq = case["B"], case["Hkv"], case["Nq"]
    s = _randn(g, B, Hkv, 1, W) * 3 + _randn(g, B, Hkv, -(-Nq // 16), W).repeat_interleave(16, dim=2)[:, :, :Nq]
    s = s + 0.5 * _randn(g, B, Hkv, Nq, W)
    return s.masked_fill(torch.arange(W, device="cuda") >= _visible(case, lens, new, W), -math.inf)


def prepare(case, seed):
    g = _gen(seed)
    lens, new = _lengths(case)
    Hkv, page = case["Hkv"], case["page"]
    need = [-(-n // page) for n in lens]
    W = max(need)
    st = dict(case=case, lens=_int(lens), new=_int(new) if case.get("ragged") else None)
    if case["op"] == "select":
        st["scores"] = _page_scores(g, case, st["lens"], _int(new), W)
        return st
    if case["op"] == "evict":
        pages, (st["table"], st["dst"]) = _tables([need, [-(-min(n, case["budget"]) // page) for n in lens]], seed)
        st["k_cache"] = _randn(g, pages, Hkv, page, case["d"]).bfloat16()
        st["v_cache"] = _randn(g, pages, Hkv, page, case["d"]).bfloat16()
        # few tokens draw most of the weight
        st["weights"] = torch.exp(2 * _randn(g, pages, Hkv, page))
        return st
    pages, (st["table"],) = _tables([need], seed)
    u = _randn(g, Hkv, case["d"])
    st["k_cache"] = _keys(g, case, pages, u)
    st["q"] = _queries(g, case, u)
    if case["op"] == "score":
        # what earlier calls left: the bounds of whole pages
        st["bounds"] = torch.stack([st["k_cache"].amin(dim=2), st["k_cache"].amax(dim=2)], dim=2)
    if case["op"] == "attn":
        st["v_cache"] = _randn(g, pages, Hkv, page, case["d"]).bfloat16()
        s = _page_scores(g, case, st["lens"], _int(new), W)
        st["blocks"] = _pick(case, s, _visible(case, st["lens"], _int(new), W))
    if case["op"] == "weights":
        st["lse"] = _lse(case, st, _int(new))
        st["weights"] = torch.rand(pages, Hkv, page, generator=g, device="cuda")
        st["out"] = torch.zeros_like(st["weights"])
    return st


def _lse(case, st, new):
    """What the attention before leaves: the log of each row's sum, -inf for padded rows."""
    B, Hq, Hkv, Nq, page, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "page", "d"))
    T = st["table"].shape[1] * page
    out = []
    for b in range(B):
        k = st["k_cache"][st["table"][b].long().clamp(min=0)].float().transpose(0, 1).reshape(Hkv, 1, T, d)
        s = (st["q"][b].float().reshape(Hkv, Hq // Hkv, Nq, d) @ k.transpose(-1, -2)) / math.sqrt(d)
        i = torch.arange(Nq, device="cuda")[:, None]
        dead = torch.arange(T, device="cuda") > i + (st["lens"][b] - new[b])
        out.append(torch.logsumexp(s.masked_fill(dead | (i >= new[b]), -math.inf), dim=-1).reshape(Hq, Nq))
    return torch.stack(out)


# ------------------------------------------------------------------ one pass

def run(state):
    return {"score": _score, "select": _select, "attn": _attn, "weights": _weights, "evict": _evict}[
        state["case"]["op"]](state)


def _new(st):
    return st["new"] if st["new"] is not None else torch.full_like(st["lens"], st["case"]["Nq"])


def _score(st):
    case = st["case"]
    if own:
        import exact_attention_69_gb300 as E
        E.kv_bounds(st["k_cache"], st["bounds"], st["table"], st["lens"], n_new=case["Nq"])
        s = E.block_scores(st["q"], st["bounds"], st["table"], st["lens"], page_size=case["page"], q_lens=st["new"])
        return {"bounds": st["bounds"], "scores": s}
    B, Hq, Hkv, Nq, d, page = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "d", "page"))
    lens, W = st["lens"].long(), st["table"].shape[1]
    # the pages that hold the newest Nq tokens; the last one again where there are fewer
    at = (lens - Nq).clamp(min=0)[:, None] // page + torch.arange((Nq + page - 2) // page + 1, device=lens.device)
    at = torch.minimum(at, (lens[:, None] - 1) // page)
    pg = st["table"].long().gather(1, at)
    k = st["k_cache"][pg].float()                                                        # [B, pages, Hkv, page, d]
    dead = (at[:, :, None] * page + torch.arange(page, device=k.device) >= lens[:, None, None])[:, :, None, :, None]
    low, high = k.masked_fill(dead, math.inf).amin(dim=3), k.masked_fill(dead, -math.inf).amax(dim=3)
    st["bounds"][pg] = torch.stack([low, high], dim=3).bfloat16()
    # the largest product that a key between the bounds can have
    b = st["bounds"][st["table"].long().clamp(min=0)].float().transpose(1, 2)            # [B, Hkv, W, 2, d]
    q = st["q"].float().reshape(B, Hkv, Hq // Hkv * Nq, d)
    s = q.clamp(max=0) @ b[:, :, :, 0].transpose(-1, -2) + q.clamp(min=0) @ b[:, :, :, 1].transpose(-1, -2)
    s = s.reshape(B, Hkv, Hq // Hkv, Nq, W).amax(dim=2) / math.sqrt(d)
    seen = _visible(case, st["lens"], _new(st), W)
    return {"bounds": st["bounds"], "scores": s.masked_fill(torch.arange(W, device=s.device) >= seen, -math.inf)}


def _pick(case, scores, seen):
    """The first and last visible pages and those of the greatest scores, ascending, then -1."""
    W = scores.shape[-1]
    i = torch.arange(W, device=scores.device)
    s = scores.masked_fill(((i < case["first"]) | (i >= seen - case["last"])) & (i < seen), math.inf)
    s = s.masked_fill(i >= seen, -math.inf)
    at = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :case["n"]]
    at = torch.where(at < seen, at, W).sort(dim=-1).values
    at = torch.nn.functional.pad(at, (0, case["n"] - at.shape[-1]), value=W)
    return torch.where(at < W, at, -1).int()


def _select(st):
    case = st["case"]
    if own:
        import exact_attention_69_gb300 as E
        return E.block_select(st["scores"], st["lens"], case["n"], page_size=case["page"], q_lens=st["new"],
                              first=case["first"], last=case["last"])
    return _pick(case, st["scores"], _visible(case, st["lens"], _new(st), st["scores"].shape[-1]))


def _attn(st):
    case = st["case"]
    if own:
        import exact_attention_69_gb300 as E
        o, lse = E.attn_blocks(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["blocks"],
                               q_lens=st["new"])
        return {"o": o, "lse": lse}
    B, Hq, Hkv, Nq, d, page, n = (case[x] for x in ("B", "Hq", "Hkv", "Nq", "d", "page", "n"))
    dev = st["q"].device
    blocks = st["blocks"].long()
    pg = st["table"].long().gather(1, blocks.clamp(min=0).reshape(B, -1)).reshape(blocks.shape)
    h = torch.arange(Hkv, device=dev)[:, None, None]
    k = st["k_cache"][pg, h].float().reshape(B, Hkv, Nq, n * page, d)                    # each query's own keys
    v = st["v_cache"][pg, h].float().reshape(B, Hkv, Nq, n * page, d)
    q = st["q"].float().reshape(B, Hkv, Hq // Hkv, Nq, d).transpose(2, 3) * (1.0 / math.sqrt(d))
    i = torch.arange(Nq, device=dev)
    new = _new(st).long()[:, None]
    last = torch.where(i < new, st["lens"].long()[:, None] - new + i, -1)[:, None, :, None, None]
    slot = blocks[..., None] * page + torch.arange(page, device=dev)                     # [B, Hkv, Nq, n, page]
    dead = ((slot > last) | (blocks[..., None] < 0)).reshape(B, Hkv, Nq, 1, n * page)
    s = (q @ k.transpose(-1, -2)).masked_fill(dead, -math.inf)                           # [B, Hkv, Nq, G, keys]
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(dim=-1, keepdim=True)
    o = torch.where(z > 0, (p @ torch.where(dead.transpose(-1, -2), 0.0, v)) / z, 0.0)
    lse = (m + torch.log(z))[..., 0]
    return {"o": o.transpose(2, 3).reshape(B, Hq, Nq, d).bfloat16(), "lse": lse.transpose(2, 3).reshape(B, Hq, Nq)}


def _weights(st):
    case = st["case"]
    if own:
        import exact_attention_69_gb300 as E
        E.kv_weights(st["q"], st["k_cache"], st["table"], st["lens"], st["lse"], st["weights"], q_lens=st["new"],
                     decay=case["decay"], out=st["out"])
        return st["out"]
    B, Hq, Hkv, Nq, d, page = (case[x] for x in ("B", "Hq", "Hkv", "Nq", "d", "page"))
    lens, new = st["lens"].long()[:, None], _new(st).long()[:, None]
    t = torch.arange(st["table"].shape[1] * page, device=lens.device)
    # slots behind the end: the last one again
    slot = torch.minimum(t, lens - 1)
    pg, at = st["table"].long().gather(1, slot // page), slot % page                     # [B, T]
    k = st["k_cache"][pg, :, at].float().transpose(1, 2)                                 # [B, Hkv, T, d]
    q = st["q"].float().reshape(B, Hkv, Hq // Hkv, Nq, d)
    s = (q @ k[:, :, None].transpose(-1, -2)) * (1.0 / math.sqrt(d))                     # [B, Hkv, G, Nq, T]
    i = torch.arange(Nq, device=t.device)
    seen = ((i < new)[:, :, None] & (slot[:, None] <= (lens - new + i)[:, :, None]))[:, None, None]
    w = torch.where(seen, torch.exp(s - st["lse"].reshape(B, Hkv, Hq // Hkv, Nq, 1)), 0.0).sum(dim=(2, 3))
    old = st["weights"][pg, :, at].transpose(1, 2) * case["decay"]                       # [B, Hkv, T]
    w = w + torch.where((slot < lens - new)[:, None], old, 0.0)
    st["out"][pg, :, at] = w.transpose(1, 2)
    return st["out"]


def _evict(st):
    case = st["case"]
    if own:
        import exact_attention_69_gb300 as E
        lens, kept = E.kv_evict(st["k_cache"], st["v_cache"], st["weights"], st["table"], st["lens"], case["budget"],
                                first=case["first"], last=case["last"], dst_table=st["dst"])
        return {"lens": lens, "kept": kept, "k_cache": st["k_cache"], "v_cache": st["v_cache"], "weights": st["weights"]}
    Hkv, page, budget = case["Hkv"], case["page"], case["budget"]
    lens = st["lens"].long()[:, None]
    t = torch.arange(st["table"].shape[1] * page, device=lens.device)
    pg = st["table"].long().clamp(min=0)[:, t // page]
    w = st["weights"][pg, :, (t % page).expand_as(pg)].transpose(1, 2)                   # [B, Hkv, T]
    w = w.masked_fill(((t < case["first"]) | (t >= lens - case["last"]))[:, None], math.inf)
    w = w.masked_fill((t >= lens)[:, None], -math.inf)
    keep = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.where(keep < lens[:, None], keep, w.shape[-1]).sort(dim=-1).values
    # places behind the new length: the last kept token again
    left = lens.clamp(max=budget)
    to = torch.minimum(torch.arange(keep.shape[-1], device=t.device), left - 1)
    src = keep.gather(2, to[:, None].expand(-1, Hkv, -1))
    h = torch.arange(Hkv, device=t.device)[:, None]
    pg = st["table"].long().gather(1, (src // page).flatten(1)).reshape(src.shape)
    dp, da = st["dst"].long().gather(1, to // page)[:, None], (to % page)[:, None]
    st["k_cache"][dp, h, da] = st["k_cache"][pg, h, src % page]
    st["v_cache"][dp, h, da] = st["v_cache"][pg, h, src % page]
    st["weights"][dp, h, da] = st["weights"][pg, h, src % page]
    kept = torch.nn.functional.pad(torch.where(keep < lens[:, None], keep, -1), (0, budget - keep.shape[-1]), value=-1)
    return {"lens": left[:, 0].int(), "kept": kept.int(), "k_cache": st["k_cache"], "v_cache": st["v_cache"],
            "weights": st["weights"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _rows(cache, pages):
    """A sequence's pages side by side: [Hkv, tokens, ...]."""
    return torch.cat([cache[p] for p in pages], dim=1).double()


def _exact_score(st, case, lens, new, table):
    page, Hkv, d, Nq = case["page"], case["Hkv"], case["d"], case["Nq"]
    bounds = st["bounds"].double()
    G = case["Hq"] // Hkv
    W = st["table"].shape[1]
    scores = torch.full((case["B"], Hkv, Nq, W), -math.inf, dtype=torch.float64, device=bounds.device)
    for b, (n, m) in enumerate(zip(lens, new)):
        for p in range(max(0, n - Nq) // page, -(-n // page)):
            k = st["k_cache"][table[b][p]][:, :min(page, n - p * page)].double()
            bounds[table[b][p]] = torch.stack([k.min(dim=1).values, k.max(dim=1).values], dim=1)
        count = -(-n // page)
        both = bounds[torch.tensor(table[b][:count], device=bounds.device)]               # [pages, Hkv, 2, d]
        for h in range(Hkv):
            q = st["q"][b, h * G:(h + 1) * G].double()                                   # [G, Nq, d]
            mid, half = both[:, h].mean(dim=1), (both[:, h, 1] - both[:, h, 0]) / 2
            s = (torch.einsum("gid,pd->gip", q, mid) + torch.einsum("gid,pd->gip", q.abs(), half)) / math.sqrt(d)
            best = s.max(dim=0).values
            for i in range(m):
                c = (n - m + i) // page + 1
                scores[b, h, i, :c] = best[i, :c]
    return {"bounds": bounds, "scores": scores}


def _exact_attn(st, case, lens, new, table):
    page, Hkv, Nq, d = case["page"], case["Hkv"], case["Nq"], case["d"]
    G = case["Hq"] // Hkv
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device=o.device)
    for b, (n, m) in enumerate(zip(lens, new)):
        pages = table[b][:-(-n // page)]
        k, v = _rows(st["k_cache"], pages), _rows(st["v_cache"], pages)
        T = k.shape[1]
        j = torch.arange(T, device=o.device)
        for lo in range(0, m, 64):  # 64 queries at a time, as a mask over all tokens
            hi = min(m, lo + 64)
            took = torch.zeros(Hkv, hi - lo, len(pages) + 1, dtype=torch.bool, device=o.device)
            took.scatter_(2, torch.where(st["blocks"][b, :, lo:hi] < 0, len(pages), st["blocks"][b, :, lo:hi]).long(), True)
            see = took[:, :, :-1].repeat_interleave(page, dim=2)
            see &= j[None] <= torch.arange(n - m + lo, n - m + hi, device=o.device)[:, None]
            s = torch.einsum("hgid,hjd->hgij", st["q"][b, :, lo:hi].double().unflatten(0, (Hkv, G)), k) / math.sqrt(d)
            s = s.masked_fill(~see[:, None], -math.inf)
            z = torch.logsumexp(s, dim=-1)
            w = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[..., None])
            o[b, :, lo:hi] = torch.einsum("hgij,hjd->hgid", w, torch.where((j < n)[:, None], v, 0.0)).flatten(0, 1)
            lse[b, :, lo:hi] = z.flatten(0, 1)
    return {"o": o, "lse": lse}


def _exact_weights(st, case, lens, new, table):
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    out = st["out"].double()
    for b, (n, m) in enumerate(zip(lens, new)):
        pages = table[b][:-(-n // page)]
        k, w = _rows(st["k_cache"], pages)[:, :n], _rows(st["weights"], pages)[:, :n] * case["decay"]
        w[:, n - m:] = 0
        for h in range(case["Hq"]):
            s = (st["q"][b, h, :m].double() @ k[h * Hkv // case["Hq"]].T) / math.sqrt(d)
            p = torch.exp(s - st["lse"][b, h, :m].double()[:, None])
            w[h * Hkv // case["Hq"]] += torch.tril(p, diagonal=n - m).sum(dim=0)
        for x, p in enumerate(pages):
            took = min(page, n - x * page)
            out[p, :, :took] = w[:, x * page:x * page + took]
    return out


def _exact_evict(st, case, lens, table):
    page, Hkv, budget = case["page"], case["Hkv"], case["budget"]
    dst = st["dst"].tolist()
    kept = torch.full((case["B"], Hkv, budget), -1, dtype=torch.int32)
    k, v, w = st["k_cache"].clone(), st["v_cache"].clone(), st["weights"].clone()
    for b, n in enumerate(lens):
        rows = torch.cat([st["weights"][p] for p in table[b][:-(-n // page)]], dim=1)[:, :n].cpu().tolist()
        m = min(n, budget)
        pt, pd = (torch.tensor(x[b], device=k.device) for x in (table, dst))
        to = torch.arange(m, device=k.device)
        for h in range(Hkv):
            sure = set(range(min(case["first"], n))) | set(range(max(0, n - case["last"]), n))
            rest = sorted((i for i in range(n) if i not in sure), key=lambda i: (-rows[h][i], i))
            take = torch.tensor(sorted(list(sure) + rest[:m - len(sure)] if n > m else range(n)))
            kept[b, h, :m] = take.int()
            take = take.to(k.device)
            for new, old in ((k, st["k_cache"]), (v, st["v_cache"]), (w, st["weights"])):
                new[pd[to // page], h, to % page] = old[pt[take // page], h, take % page]
    return {"lens": _int([min(n, budget) for n in lens]), "kept": kept.to(k.device), "k_cache": k.double(),
            "v_cache": v.double(), "weights": w.double()}


def _exact_select(st, case, lens, new):
    out = torch.full((case["B"], case["Hkv"], case["Nq"], case["n"]), -1, dtype=torch.int32)
    scores = st["scores"].double().cpu().tolist()
    for b, (n, m) in enumerate(zip(lens, new)):
        for h in range(case["Hkv"]):
            for i in range(m):
                c, row = (n - m + i) // case["page"] + 1, scores[b][h][i]
                sure = [x for x in range(c) if x < case["first"] or x >= c - case["last"]]
                rest = sorted((x for x in range(case["first"], c - case["last"])), key=lambda x: (-row[x], x))
                took = sorted(sure + rest[:case["n"] - len(sure)])
                out[b, h, i, :len(took)] = torch.tensor(took, dtype=torch.int32)
    return out.cuda()


def exact(case, seed):
    st = prepare(case, seed)
    lens, new = _lengths(case)
    if case["op"] == "select":
        return _exact_select(st, case, lens, new)
    table = st["table"].tolist()
    if case["op"] == "evict":
        return _exact_evict(st, case, lens, table)
    return {"score": _exact_score, "attn": _exact_attn, "weights": _exact_weights}[case["op"]](st, case, lens, new, table)
