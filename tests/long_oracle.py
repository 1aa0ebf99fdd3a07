"""Plain 64-bit definitions (CPU, torch float64) of the long-cache operators, with the
error bounds of the kernels' roundings.

Bounds, per element, with T = 2^-24 (half an fp32 step) and U = 2^-8 (half a bf16 step):
  scores     a sum of 2 d products that are exact in fp32, added in fp32 in any order with
             either rounding: (2 d + 4) 2 T of the sum of their magnitudes. The largest
             over heads moves by no more than the largest bound.
  weights    exp(scale q . k - lse): the exponent is off by (d + 4) 2 T scale sum |q k| and by
             2 T of its own size, exp2 adds 2^-21, so each term moves relatively by the
             sum of these; n terms added in fp32: n T of their sum; with the old weight's
             product one more step.
  attention  as in cache_oracle: P is rounded to bf16, U sum p |v|; scores (d + 2) 2 T scale
             sum |q k|; then U |o|.
Pages chosen and tokens kept are exact.
"""
import math

import torch

U = 2.0 ** -8
T = 2.0 ** -24


def lengths(p_lens, q_lens, Nq, most):
    lens = [max(0, min(int(n), most)) for n in p_lens]
    new = [Nq] * len(lens) if q_lens is None else [max(0, min(Nq, int(n))) for n in q_lens]
    return lens, new


def seen(n, m, i, mask):
    """Slots that query i of m sees of n."""
    if i >= m:
        return 0
    return max(0, min(n, n - m + i + 1)) if mask == "causal_br" else n


def rows(cache, pages, n):
    """The first n tokens of a sequence: [Hk, n, ...] float64; zeros where no page is named."""
    page = cache.shape[2]
    out = torch.zeros(cache.shape[1], n, *cache.shape[3:], dtype=torch.float64)
    for x in range(-(-n // page)):
        pg, took = int(pages[x]), min(page, n - x * page)
        if 0 <= pg < cache.shape[0]:
            out[:, x * page:x * page + took] = cache[pg, :, :took].double()
    return out


def bounds(k_cache, before, table, lens, n_new):
    out = before.clone()
    page = k_cache.shape[2]
    for b, n in enumerate(lengths(lens, None, 0, table.shape[1] * page)[0]):
        for x in range(0 if n_new is None else max(0, n - n_new) // page, -(-n // page)):
            pg, took = int(table[b, x]), min(page, n - x * page)
            if 0 <= pg < k_cache.shape[0] and n_new != 0:
                k = k_cache[pg, :, :took].double()
                out[pg] = torch.stack([k.amin(1), k.amax(1)], 1).to(torch.bfloat16)
    return out


def scores(q, bnd, table, lens, q_lens, page, scale, mask):
    """(scores, bound)"""
    B, Hq, Nq, d = q.shape
    Hk, W = bnd.shape[1], table.shape[1]
    G = Hq // Hk
    out = torch.full((B, Hk, Nq, W), -math.inf, dtype=torch.float64)
    err = torch.zeros_like(out)
    lens, new = lengths(lens, q_lens, Nq, W * page)
    for b in range(B):
        for x in range(-(-lens[b] // page)):
            pg = int(table[b, x])
            lo, hi = (bnd[pg, :, s].double() for s in (0, 1)) if 0 <= pg < bnd.shape[0] else (torch.zeros(Hk, d).double(),) * 2
            qq = q[b].double().reshape(Hk, G, Nq, d)
            neg, pos = qq.clamp(max=0) * lo[:, None, None], qq.clamp(min=0) * hi[:, None, None]
            s, e = scale * (neg + pos).sum(-1).amax(1), scale * (neg.abs() + pos.abs()).sum(-1).amax(1)
            for i in range(Nq):
                if x * page < seen(lens[b], new[b], i, mask):
                    out[b, :, i, x], err[b, :, i, x] = s[:, i], e[:, i]
    return out, (2 * d + 4) * 2 * T * err


def take(values, n, first, last):
    """Indices of the n chosen of a list: the first and last for sure, then the greatest
    (NaN above all), ties to the lowest; ascending."""
    if len(values) <= n:
        return list(range(len(values)))
    sure = list(range(first)) + list(range(len(values) - last, len(values)))
    rest = range(first, len(values) - last)
    order = sorted(rest, key=lambda x: (0, 0.0, x) if math.isnan(values[x]) else (1, -values[x], x))
    return sorted(sure + order[:n - first - last])


def select(s, lens, q_lens, n, page, first, last, mask):
    B, Hk, Nq, W = s.shape
    out = torch.full((B, Hk, Nq, n), -1, dtype=torch.int32)
    lens, new = lengths(lens, q_lens, Nq, W * page)
    for b in range(B):
        for h in range(Hk):
            for i in range(Nq):
                c = min(W, -(-seen(lens[b], new[b], i, mask) // page))
                got = take(s[b, h, i, :c].tolist(), n, first, last)
                out[b, h, i, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


def blocks(q, k_cache, v_cache, table, lens, lists, q_lens, scale, mask):
    """(o, bound, lse, bound)"""
    B, Hq, Nq, d = q.shape
    Hk, page, W = k_cache.shape[1], k_cache.shape[2], table.shape[1]
    G = Hq // Hk
    lens, new = lengths(lens, q_lens, Nq, W * page)
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    for b in range(B):
        k, v = rows(k_cache, table[b], lens[b]), rows(v_cache, table[b], lens[b])
        for i in range(new[b]):
            n = seen(lens[b], new[b], i, mask)
            for h in range(Hk):
                named = sorted({int(x) for x in lists[b, h, i].tolist() if 0 <= x < W})
                at = torch.tensor([t for x in named for t in range(x * page, min(n, (x + 1) * page))], dtype=torch.long)
                if len(at) == 0:
                    continue
                hs = slice(h * G, (h + 1) * G)
                qq, kk, vv = q[b, hs, i].double(), k[h, at], v[h, at]
                s = scale * (qq @ kk.T)
                err = (d + 2) * 2 * T * scale * (qq.abs() @ kk.abs().T).amax(-1)
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None])
                o[b, hs, i] = w @ vv
                ob[b, hs, i] = U * (w @ vv).abs() + (U + 2 * err + 2.0 ** -21)[:, None] * (w @ vv.abs())
                lse[b, hs, i] = z
                lb[b, hs, i] = err + 2.0 ** -20 * (1 + z.abs())
    return o, ob, lse, lb


def blocks_two_parts(q, k_cache, v_cache, table, lens, lists, q_lens, scale, mask, most):
    """(o, bound) where P is held in two bf16 parts: the second is the first's rounding, rounded
    itself, U of U p. What is left, with z = sum p |v|: U |o| of the output; U^2 z; the score's error
    twice and exp2's, as above; products of up to `most` slots, added in fp32 with either
    rounding, and 8 more steps for the join and the division: (most + 8) 2 T z."""
    o, _, lse, lb = blocks(q, k_cache, v_cache, table, lens, lists, q_lens, scale, mask)
    z = blocks(q, k_cache, v_cache.abs(), table, lens, lists, q_lens, scale, mask)[0]
    err = torch.where(lse == -math.inf, 0.0, lb - 2.0 ** -20 * (1 + lse.abs()))[..., None]
    return o, U * o.abs() + (U * U + 2 * err + 2.0 ** -21 + (most + 8) * 2 * T) * z


def weights(q, k_cache, table, lens, lse, before, q_lens, scale, mask, decay, out=None):
    """(weights, bound); `before` and the result as [n_pages, Hk, page]."""
    B, Hq, Nq, d = q.shape
    Hk, page, W = k_cache.shape[1], k_cache.shape[2], table.shape[1]
    G = Hq // Hk
    lens, new = lengths(lens, q_lens, Nq, W * page)
    res = (before if out is None else out).double().clone()
    err = torch.zeros_like(res)
    for b in range(B):
        n, m = lens[b], new[b]
        k = rows(k_cache, table[b], n)
        old = rows(before, table[b], n) * decay if decay else torch.zeros(Hk, n, dtype=torch.float64)
        if mask == "causal_br":
            old[:, max(0, n - m):] = 0.0
        w, e = torch.zeros(Hk, n, dtype=torch.float64), torch.zeros(Hk, n, dtype=torch.float64)
        for i in range(m):
            c = seen(n, m, i, mask)
            for h in range(Hq):
                z = float(lse[b, h, i])
                if z == -math.inf or c == 0:
                    continue
                kk, qq = k[h // G, :c], q[b, h, i].double()
                a = scale * (kk @ qq) - z
                p = torch.exp(a)
                w[h // G, :c] += p
                rel = (d + 4) * 2 * T * scale * (kk.abs() @ qq.abs()) + 2 * T * a.abs() + 2.0 ** -21
                e[h // G, :c] += p * torch.where(p == 0, 0.0, rel)
        terms = m * G + 2
        e = e + terms * T * (w + old)
        w = w + old
        for x in range(-(-n // page)):
            pg, took = int(table[b, x]), min(page, n - x * page)
            if 0 <= pg < k_cache.shape[0]:
                res[pg, :, :took] = w[:, x * page:x * page + took]
                err[pg, :, :took] = e[:, x * page:x * page + took]
    return res, err


def evict(k_cache, v_cache, wts, table, lens, budget, first, last, dst=None):
    """(k, v, weights, new lengths, kept); sources that no page holds read as zeros."""
    n_pages, Hk, page = wts.shape
    to = table if dst is None else dst
    lens, _ = lengths(lens, None, 0, table.shape[1] * page)
    caches = (k_cache, v_cache, wts)
    out = [c.clone() for c in caches]
    kept = torch.full((len(lens), Hk, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(Hk):
            got = take(rows(wts, table[b], n)[h].tolist(), budget, first, last)
            kept[b, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
            for x, src in enumerate(got):
                pd = int(to[b, x // page]) if x // page < to.shape[1] else -1
                if not 0 <= pd < n_pages or (dst is None and x == src):
                    continue
                ps = int(table[b, src // page])
                for new, old in zip(out, caches):
                    new[pd, h, x % page] = old[ps, h, src % page] if 0 <= ps < n_pages else 0
    return (*out, torch.tensor([min(n, budget) for n in lens], dtype=torch.int32), kept)
