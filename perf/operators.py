"""The cache operators as they are measured: cases, inputs, plain forms and the
framework's calls.

    attn_paged     attention of a batch of sequences over a paged key/value
                   cache: a prefix that all of them share, then each one's own
                   pages
    qk_norm_rope   root-mean-square norm of every query and key head with the
                   rotary position embedding in the same pass, and its gradient
    kv_append      new keys and values into their pages, keys (and queries)
                   normed and rotated on the way

Where `own` is false, run() computes an operator from elementary torch
operations in 32 bits (angles in 64); where it is true, it calls the framework.
exact() is the definition in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The smallest call of a chat server: four conversations over a short
        # system prompt, one new token each. Latency is all that counts.
        dict(name="decode few", op="attn", B=4, Hq=16, Hkv=4, d=64, Nq=1, P=512, lo=1, hi=160, page=16, ragged=False,
             shape=1),
        # An ordinary decoding step: 32 conversations, a prompt of 4096 tokens.
        dict(name="decode", op="attn", B=32, Hq=32, Hkv=8, d=128, Nq=1, P=4096, lo=64, hi=1024, page=16, ragged=False,
             shape=2),
        # A large one: many requests over the same long document.
        dict(name="decode long", op="attn", B=96, Hq=32, Hkv=8, d=128, Nq=1, P=32768, lo=256, hi=2048, page=64,
             ragged=False, shape=3),
        # Checking five drafted tokens per sequence; odd counts of heads, a
        # prefix that ends inside a page, ragged numbers of drafted tokens.
        dict(name="verify", op="attn", B=7, Hq=15, Hkv=5, d=64, Nq=5, P=1021, lo=5, hi=700, page=32, ragged=True,
             shape=4),
        # A chunk of each prompt behind a shared prefix (prefill by chunks).
        dict(name="chunk", op="attn", B=3, Hq=16, Hkv=16, d=128, Nq=512, P=2048, lo=512, hi=1500, page=128,
             ragged=True, shape=5),
        # No shared prefix, one key head for all queries, sequences from nothing
        # (an idle slot) to 4096 tokens.
        dict(name="decode alone", op="attn", B=16, Hq=8, Hkv=1, d=32, Nq=1, P=0, lo=0, hi=4096, page=256, ragged=False,
             shape=6),
        # A training step of a causal language model, grouped keys.
        dict(name="norm train", op="norm", B=4, Hq=16, Hkv=4, N=2048, d=128, rot=128, interleaved=False, fused=False,
             far=0, train=True),
        # A short odd batch: 77 tokens, half of each head rotated, pairs side by side.
        dict(name="norm train odd", op="norm", B=2, Hq=5, Hkv=5, N=77, d=64, rot=32, interleaved=True, fused=False,
             far=1000, train=True),
        # The largest training step: views of one fused projection.
        dict(name="norm train large", op="norm", B=8, Hq=32, Hkv=8, N=4096, d=128, rot=128, interleaved=False,
             fused=True, far=0, train=True),
        # A long prompt, forward only, positions far out.
        dict(name="norm long", op="norm", B=1, Hq=8, Hkv=8, N=16384, d=128, rot=128, interleaved=False, fused=True,
             far=100000, train=False),
        # The appending half of a decoding step: 32 sequences, one token each.
        dict(name="append decode", op="append", B=32, Hq=32, Hkv=8, N=1, d=128, rot=128, interleaved=False, norm=True,
             P=4096, lo=64, hi=1024, page=16, ragged=False, shape=7),
        # A ragged batch of prompt chunks, no norm, pairs side by side.
        dict(name="append chunk", op="append", B=5, Hq=16, Hkv=4, N=1000, d=64, rot=64, interleaved=True, norm=False,
             P=1021, lo=1, hi=900, page=64, ragged=True, shape=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_attn(rng):
    d = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    Nq = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 512)])
    P = rng.choice([0, _log(rng, 1, 32768), _log(rng, 256, 32768), _log(rng, 256, 32768)])
    hi = _log(rng, max(Nq, 16), 4096)
    return dict(op="attn", B=_log(rng, 1, 96), Hq=Hkv * G, Hkv=Hkv, d=d, Nq=Nq, P=P, lo=rng.choice([Nq, Nq, hi]), hi=hi,
                page=rng.choice([16, 32, 64, 128, 256]), ragged=Nq > 1 and rng.random() < 0.5,
                shape=rng.randrange(1 << 20))


def _draw_norm(rng):
    d = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    return dict(op="norm", B=_log(rng, 1, 8), Hq=Hkv * rng.choice([1, 2, 3, 4, 7]), Hkv=Hkv, N=_log(rng, 1, 16384), d=d,
                rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                far=rng.choice([0, 1000, 100000, 1000000]), train=rng.random() < 0.6)


def _draw_append(rng):
    d = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    N = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
    return dict(op="append", B=_log(rng, 1, 96), Hq=Hkv * rng.choice([1, 2, 3, 4, 7, 8]), Hkv=Hkv, N=N, d=d,
                rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.5,
                P=rng.choice([0, _log(rng, 1, 100000)]), lo=0, hi=_log(rng, 8, 4096),
                page=rng.choice([16, 32, 64, 128, 256]), ragged=N > 1 and rng.random() < 0.5,
                shape=rng.randrange(1 << 20))


def draw(rng):
    """One more case, no dearer than the largest listed one of its operator."""
    make = rng.choice([_draw_attn, _draw_attn, _draw_norm, _draw_append])
    while True:
        case = make(rng)
        top = [work(c) for c in listed() if c["op"] == case["op"]]
        w = work(case)
        if case["op"] == "append" and _tokens(case) * case["Hkv"] * case["d"] > (1 << 25):
            continue  # a cache of this size is copied and compared whole
        if all(w[m] <= max(t[m] for t in top) for m in ("bytes", "flops")):
            return case


def _own_lengths(case):
    """Tokens that each sequence holds in its own pages, spread over [lo, hi]; and
    how many of the new tokens of each are real. From the case alone."""
    r = random.Random(case["shape"])
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + int(round((hi - lo) * r.random() ** 1.5)) for _ in range(B)]
    lens[r.randrange(B)] = hi
    if B > 1 and lo == 0:
        lens[lens.index(min(lens))] = 0
    n = case.get("Nq", case.get("N"))
    new = [r.randint(1, n) if case["ragged"] else n for _ in range(B)]
    return lens, new


def _attn_lengths(case):
    lens, new = _own_lengths(case)
    if case["Nq"] > 1:
        lens = [max(a, b) for a, b in zip(lens, new)]  # the new tokens are in the cache already
    return lens, new


def _tokens(case):
    """Tokens that the pages of an append case hold."""
    lens, _ = _own_lengths(case)
    return sum(-(-(n + case["N"]) // case["page"]) * case["page"] for n in lens)


def work(case):
    d = case["d"]
    if case["op"] == "attn":
        B, Hq, Hkv, Nq, P = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "P"))
        lens, new = _attn_lengths(case)
        pairs = 0
        for n, m in zip(lens, new):  # row i of m sees the keys up to i + (P + n) - m
            first = P + n - m + 1
            pairs += sum(max(0, first + i) for i in range(m))
        kv = 2 * 2 * Hkv * d * (P + sum(lens))
        tables = 4 * (-(-P // case["page"]) + sum(-(-n // case["page"]) for n in lens) + 2 * B)
        return dict(bytes=2 * 2 * B * Hq * Nq * d + 4 * B * Hq * Nq + kv + tables, flops=4 * d * Hq * pairs)
    if case["op"] == "norm":
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hkv"])
        side = 8 * case["B"] * case["N"] + 4 * case["rot"] + 4 * 2 * d
        fwd = 2 * 2 * rows * d + side
        bwd = 3 * 2 * rows * d + side
        flops = rows * (4 * d + 3 * case["rot"])
        if case["train"]:
            return dict(bytes=fwd + bwd, flops=flops + rows * (9 * d + 3 * case["rot"]))
        return dict(bytes=fwd, flops=flops)
    B, N, Hq, Hkv = (case[k] for k in ("B", "N", "Hq", "Hkv"))
    _, new = _own_lengths(case)
    rows = B * N * Hq + sum(new) * Hkv
    return dict(bytes=2 * 2 * (B * N * Hq + 2 * sum(new) * Hkv) * d + 4 * 3 * B + 4 * case["rot"],
                flops=rows * (3 * case["rot"] + (4 * d if case["norm"] else 0)))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFFFFFF)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _pages(case, lens, extra, seed):
    """Block table [B, max pages] over shuffled pages; unused entries are -1."""
    page = case["page"]
    need = [-(-(n + extra) // page) for n in lens]
    first = -(-case["P"] // page) if case["op"] == "attn" else 0
    total = first + sum(need)
    order = list(range(total))
    random.Random(seed).shuffle(order)
    prefix, at = order[:first], first
    table = []
    width = max(1, max(need))
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return max(1, total), prefix, table


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _freqs(rot):
    return BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def prepare(case, seed):
    g = _gen(seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "attn":
        lens, new = _attn_lengths(case)
        pages, prefix, table = _pages(case, lens, 0, seed)
        shape = (pages, Hkv, case["page"], d)
        # queries and keys share a direction per key head, as trained heads do;
        # the first tokens of the prefix draw more of the attention
        u = _randn(g, Hkv, 1, d)
        q = _randn(g, B, Hkv, Hq // Hkv, case["Nq"], d) + 0.3 * u[:, None]
        k = _randn(g, *shape) + 0.3 * u
        if prefix:
            k[prefix[0], :, :4] += 1.5 * u
        return dict(case=case, q=q.reshape(B, Hq, case["Nq"], d).bfloat16(), k_cache=k.bfloat16(),
                    v_cache=_randn(g, *shape).bfloat16(), table=_int(table), lens=_int(lens),
                    new=_int(new) if case["ragged"] else None, prefix=_int(prefix) if prefix else None)
    if case["op"] == "norm":
        N = case["N"]
        # one channel in sixteen is an outlier, as in trained projections
        gain = torch.where(torch.arange(d, device="cuda") % 16 == 3, 6.0, 1.0)
        if case["fused"]:  # the projection's output [B, N, heads, d], queries and keys side by side
            x = (_randn(g, B, N, Hq + Hkv, d) * gain).bfloat16()
            q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
        else:
            q = (_randn(g, B, Hq, N, d) * gain).bfloat16()
            k = (_randn(g, B, Hkv, N, d) * gain).bfloat16()
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        st = dict(case=case, q=q, k=k, wq=(1 + 0.2 * _randn(g, d)).bfloat16(), wk=(1 + 0.2 * _randn(g, d)).bfloat16(),
                  pos=start + torch.arange(N, device="cuda"), freqs=_freqs(case["rot"]))
        if case["train"]:
            st["dq"], st["dk"] = _randn(g, B, Hq, N, d).bfloat16(), _randn(g, B, Hkv, N, d).bfloat16()
            for n in ("q", "k", "wq", "wk"):
                st[n].requires_grad_(True)
        return st
    lens, new = _own_lengths(case)
    N = case["N"]
    pages, _, table = _pages(case, lens, N, seed)
    shape = (pages, Hkv, case["page"], d)
    # the fused projection's output [B, N, queries | keys | values, d]
    x = _randn(g, B, N, Hq + 2 * Hkv, d).bfloat16()
    return dict(case=case, q=x[:, :, :Hq].transpose(1, 2), k=x[:, :, Hq:Hq + Hkv].transpose(1, 2),
                v=x[:, :, Hq + Hkv:].transpose(1, 2), k_cache=_randn(g, *shape).bfloat16(),
                v_cache=_randn(g, *shape).bfloat16(), table=_int(table), starts=_int(lens),
                counts=_int(new) if case["ragged"] else None, freqs=_freqs(case["rot"]),
                wq=(1 + 0.2 * _randn(g, d)).bfloat16() if case["norm"] else None,
                wk=(1 + 0.2 * _randn(g, d)).bfloat16() if case["norm"] else None)


# ------------------------------------------------------------------ one pass

def run(state):
    return {"attn": _attn, "norm": _norm, "append": _append}[state["case"]["op"]](state)


def _attn(st):
    case = st["case"]
    if own:
        import exact_attention_69_gb300 as E
        o, lse = E.attn_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], q_lens=st["new"],
                              prefix_table=st["prefix"], prefix_len=case["P"])
        return {"o": o, "lse": lse}
    B, Hq, Hkv, d, Nq, P, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "Nq", "P", "page"))
    dev = st["q"].device
    G = Hq // Hkv
    q = st["q"].float().reshape(B, Hkv, G * Nq, d) * (1.0 / math.sqrt(d))
    lens = st["lens"].long()
    new = st["new"].long() if st["new"] is not None else torch.full_like(lens, Nq)
    # keys that row i of sequence b sees, counted from the prefix's first
    i = torch.arange(Nq, device=dev)
    seen = torch.where(i < new[:, None], (P + lens - new)[:, None] + i + 1, 0)          # [B, Nq]
    seen = seen[:, None, None, :].expand(B, Hkv, G, Nq).reshape(B, Hkv, G * Nq, 1)
    # the sequences' own keys, gathered from their pages
    t = torch.arange(st["table"].shape[1] * page, device=dev)
    pg = st["table"].long().clamp(min=0)[:, t // page]                                   # [B, T]
    live = (t < lens[:, None])[:, None, :, None]
    k = torch.where(live, st["k_cache"][pg, :, (t % page).expand(B, -1)].float().transpose(1, 2), 0.0)
    v = torch.where(live, st["v_cache"][pg, :, (t % page).expand(B, -1)].float().transpose(1, 2), 0.0)
    s = q @ k.transpose(-1, -2)
    s = s.masked_fill((P + t >= seen) | (t >= lens[:, None, None, None]), -math.inf)
    if P:  # the shared prefix: one set of keys for the rows of every sequence
        tp = torch.arange(P, device=dev)
        pp = st["prefix"].long()[tp // page]
        kp = st["k_cache"][pp, :, tp % page].float().transpose(0, 1)                     # [Hkv, P, d]
        vp = st["v_cache"][pp, :, tp % page].float().transpose(0, 1)
        rows = q.transpose(0, 1).reshape(Hkv, B * G * Nq, d)
        sp = (rows @ kp.transpose(-1, -2)).reshape(Hkv, B, G * Nq, P).transpose(0, 1)
        s = torch.cat([sp.masked_fill(tp >= seen, -math.inf), s], dim=-1)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(dim=-1, keepdim=True)
    o = p[..., P:] @ v
    if P:
        pr = p[..., :P].transpose(0, 1).reshape(Hkv, B * G * Nq, P)
        o = o + (pr @ vp).reshape(Hkv, B, G * Nq, d).transpose(0, 1)
    o = torch.where(z > 0, o / z, 0.0)
    return {"o": o.reshape(B, Hq, Nq, d).bfloat16(), "lse": (m + torch.log(z)).reshape(B, Hq, Nq)}


def _angles(pos, freqs):
    """cos and sin of the positions' angles: products in 64 bits, then 32."""
    a = pos[..., None].double() * freqs
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, c, s, rot, interleaved):
    """The first `rot` channels of x turned by the angles, in 32 bits."""
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _rms(x):
    return torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)


def _norm_back(x, w, dy, c, s, rot, interleaved):
    """Gradients of turn(x * rms(x) * w) with respect to x and w."""
    r = _rms(x)
    g = _turn(dy, c, -s, rot, interleaved)          # back through the turn
    h = g * w
    dx = r * h - x * (r * r * r) * (h * x).mean(dim=-1, keepdim=True)
    return dx.bfloat16(), (g * x * r).sum(dim=(0, 1, 2)).bfloat16()


def _norm(st):
    case = st["case"]
    rot, il = case["rot"], case["interleaved"]
    if own:
        import exact_attention_69_gb300 as E
        how = dict(inv_freq=st["freqs"], positions=st["pos"], interleaved=il, eps=EPS)
        if not case["train"]:
            q, k = E.qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], **how)
            return {"q": q, "k": k}
        q, k = E.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], **how)
        dq, dk, dwq, dwk = torch.autograd.grad((q, k), (st["q"], st["k"], st["wq"], st["wk"]), (st["dq"], st["dk"]))
        return {"q": q.detach(), "k": k.detach(), "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    with torch.no_grad():
        c, s = (a[:, None] for a in _angles(st["pos"], st["freqs"]))
        q, k, wq, wk = (st[n].float() for n in ("q", "k", "wq", "wk"))
        out = {"q": _turn(q * _rms(q) * wq, c, s, rot, il).bfloat16(),
               "k": _turn(k * _rms(k) * wk, c, s, rot, il).bfloat16()}
        if case["train"]:
            out["dq"], out["dwq"] = _norm_back(q, wq, st["dq"].float(), c, s, rot, il)
            out["dk"], out["dwk"] = _norm_back(k, wk, st["dk"].float(), c, s, rot, il)
        return out


def _append(st):
    case = st["case"]
    B, N, P, page = case["B"], case["N"], case["P"], case["page"]
    rot, il = case["rot"], case["interleaved"]
    if own:
        import exact_attention_69_gb300 as E
        q = E.kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["starts"],
                        counts=st["counts"], position_offset=P, inv_freq=st["freqs"], interleaved=il,
                        eps=EPS if case["norm"] else None, k_weight=st["wk"], q=st["q"], q_weight=st["wq"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    dev = st["k"].device
    n = torch.arange(N, device=dev)
    slot = st["starts"].long()[:, None] + n                                              # [B, N]
    c, s = (a[:, None] for a in _angles(P + slot, st["freqs"]))
    q, k = st["q"].float(), st["k"].float()
    if case["norm"]:
        q, k = q * _rms(q) * st["wq"].float(), k * _rms(k) * st["wk"].float()
    k = _turn(k, c, s, rot, il).bfloat16().transpose(1, 2)                               # [B, N, Hkv, d]
    v = st["v"].transpose(1, 2)
    pg, at = st["table"].long().gather(1, slot // page), slot % page
    if st["counts"] is not None:  # tokens behind a sequence's count leave the cache as it was
        real = (n < st["counts"].long()[:, None])[:, :, None, None]
        k = torch.where(real, k, st["k_cache"][pg, :, at])
        v = torch.where(real, v, st["v_cache"][pg, :, at])
    st["k_cache"][pg, :, at] = k
    st["v_cache"][pg, :, at] = v
    return {"q": _turn(q, c, s, rot, il).bfloat16(), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_attn(st, case):
    B, Hq, Hkv, Nq, P, page = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "P", "page"))
    lens, new = _attn_lengths(case)
    if not case["ragged"]:
        new = [Nq] * B
    table = st["table"].tolist()
    pre = st["prefix"].tolist() if P else []

    def rows(cache, pages, n):
        got = torch.cat([cache[p] for p in pages], dim=1)[:, :n] if n else cache[0][:, :0]
        return got.double()

    kp, vp = (rows(st[c], pre, P) for c in ("k_cache", "v_cache"))
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device=st["q"].device)
    for b in range(B):
        n, used = lens[b], -(-lens[b] // page)
        k = torch.cat([kp, rows(st["k_cache"], table[b][:used], n)], dim=1).repeat_interleave(Hq // Hkv, dim=0)
        v = torch.cat([vp, rows(st["v_cache"], table[b][:used], n)], dim=1).repeat_interleave(Hq // Hkv, dim=0)
        total = P + n
        if total == 0:
            continue
        m = new[b]
        s = torch.einsum("hid,hjd->hij", st["q"][b, :, :m].double(), k) / math.sqrt(case["d"])
        i = torch.arange(m, device=s.device)[:, None]
        j = torch.arange(total, device=s.device)[None, :]
        s = s.where(j <= i + (total - m), torch.tensor(-math.inf, dtype=torch.float64, device=s.device))
        some = (i + (total - m) >= 0).expand(m, 1)[:, 0]
        s = s[:, some]
        o[b, :, :m][:, some] = torch.einsum("hij,hjd->hid", torch.softmax(s, dim=-1), v)
        lse[b, :, :m][:, some] = torch.logsumexp(s, dim=-1)
    return {"o": o, "lse": lse}


def _complex_turn(x, pos, freqs, rot, interleaved):
    """The turn as a product of complex numbers, in 64 bits."""
    a = pos.double()[:, None, :, None] * freqs
    z = torch.polar(torch.ones_like(a), a)
    r = x[..., :rot]
    pair = r.unflatten(-1, (rot // 2, 2)) if interleaved else r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    y = y if interleaved else y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., rot:]], dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(st, case)
    rot, il = case["rot"], case["interleaved"]

    def normed(x, w):
        return x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w

    if case["op"] == "norm":
        out = {}
        for n in ("q", "k"):
            parts = [st[n].detach()]  # one sequence at a time: the gradient's graph is in 64 bits
            w = st["w" + n].detach().double().requires_grad_(case["train"])
            ys, gs, gw = [], [], torch.zeros_like(w)
            for b in range(case["B"]):
                x = parts[0][b:b + 1].double().requires_grad_(case["train"])
                y = _complex_turn(normed(x, w), st["pos"][b:b + 1], st["freqs"], rot, il)
                if case["train"]:
                    dx, dw = torch.autograd.grad(y, (x, w), st["d" + n][b:b + 1].double())
                    gs.append(dx)
                    gw = gw + dw
                ys.append(y.detach())
            out[n] = torch.cat(ys)
            if case["train"]:
                out["d" + n], out["dw" + n] = torch.cat(gs), gw.detach()
        return {n: out[n] for n in (("q", "k", "dq", "dk", "dwq", "dwk") if case["train"] else ("q", "k"))}
    q, k = st["q"].double(), st["k"].double()
    if case["norm"]:
        q, k = normed(q, st["wq"].double()), normed(k, st["wk"].double())
    lens, new = _own_lengths(case)
    pos = case["P"] + st["starts"].long()[:, None] + torch.arange(case["N"], device=q.device)
    q, k = (_complex_turn(x, pos, st["freqs"], rot, il) for x in (q, k))
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    table = st["table"].tolist()
    page = case["page"]
    for b in range(case["B"]):
        done = 0
        while done < new[b]:  # one page of the sequence at a time
            at = lens[b] + done
            step = min(new[b] - done, page - at % page)
            there = slice(at % page, at % page + step)
            kc[table[b][at // page]][:, there] = k[b, :, done:done + step]
            vc[table[b][at // page]][:, there] = st["v"][b, :, done:done + step].double()
            done += step
    return {"q": q, "k_cache": kc, "v_cache": vc}
