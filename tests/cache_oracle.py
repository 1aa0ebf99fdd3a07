"""Plain 64-bit definitions (CPU, torch float64) of the norm with rotation, the
cache append and paged attention, with the error bounds of the kernels' roundings.

Bounds, per element, with u = 2^-8 (half a bf16 step relative to the value):
  rotation    y is formed in fp32 from a pair (a, b): the cosine and sine are within
              2^-22, products and the norm add a few units of 2^-24, so the error
              before the last rounding is at most 2^-19 (|a| + |b|); then u |y|.
  gradient    dx = r h - x r^3 mean(h x), fp32: 2^-19 of the sum of the magnitudes of
              its terms; then u |dx|. dw: n terms added in fp32, n 2^-24 sum |term| at
              most, and 2^-19 of each term; then half a step of its type.
  attention   P is rounded to bf16 before the second product: u sum p |v|. The scores
              are fp32 sums of d products: (d + 2) 2^-24 scale sum |q k|, which moves
              p relatively by as much; exp2 adds 2^-22. Then u |o|. The LSE moves by the
              largest score's error, plus 2^-20 for exp2, log2 and the sum.
"""
import math

import torch

U = 2.0 ** -8
T = 2.0 ** -24


def rotate(x, pos, freqs, interleaved, back=False):
    """x [B, H, N, d] float64; pos [B, N]; returns (y, |a| + |b| of each pair)."""
    if freqs is None:
        return x.clone(), x.abs()
    rot = 2 * len(freqs)
    ang = pos.to(torch.float64)[:, None, :, None] * freqs
    c, s = torch.cos(ang), torch.sin(ang) * (-1.0 if back else 1.0)
    y, mag = x.clone(), x.abs()
    if interleaved:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    else:
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    a, b = x[..., i], x[..., j]
    y[..., i] = a * c - b * s
    y[..., j] = a * s + b * c
    mag[..., i] = mag[..., j] = a.abs() + b.abs()
    return y, mag


def norm_rope(x, w, pos, freqs, interleaved, eps):
    """(y, bound) of one of q and k; x bf16 or float64, w any float or None."""
    x = x.double()
    if eps is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        x = x * (1.0 if w is None else w.double())
    y, mag = rotate(x, pos, freqs, interleaved)
    return y, U * y.abs() + 2.0 ** -19 * mag


def norm_rope_back(x, w, dy, pos, freqs, interleaved, eps):
    """(dx, bound, dw, bound): the formula's gradients."""
    x, dy = x.double(), dy.double()
    g, mag = rotate(dy, pos, freqs, interleaved, back=True)
    if eps is None:
        return g, U * g.abs() + 2.0 ** -19 * mag, None, None
    wd = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h = g * wd
    dx = r * h - x * r ** 3 * (h * x).mean(-1, keepdim=True)
    hm = mag * wd.abs()
    terms = r * hm + x.abs() * r ** 3 * (hm * x.abs()).mean(-1, keepdim=True)
    t = g * x * r
    n = x.shape[0] * x.shape[1] * x.shape[2]
    dw, big = t.sum((0, 1, 2)), (mag * x.abs() * r).sum((0, 1, 2))
    half = torch.finfo(w.dtype).eps / 2 if w is not None else 0.0
    return (dx, U * dx.abs() + 2.0 ** -19 * terms, dw,
            half * dw.abs() + (n * T + 2.0 ** -19) * big)


def append(k, v, k_cache, v_cache, table, starts, counts, pos, freqs, interleaved, eps, wk):
    """Caches after the append, float64, and the bound of the key cache."""
    B, Hk, N, d = k.shape
    page = k_cache.shape[2]
    y, bound = norm_rope(k, wk, pos, freqs, interleaved, eps)
    kc, vc = k_cache.double().clone(), v_cache.double().clone()
    kb = torch.zeros_like(kc)
    for b in range(B):
        if starts[b] < 0:
            continue
        for n in range(N if counts is None else min(N, int(counts[b]))):
            slot = int(starts[b]) + n
            if slot // page >= table.shape[1]:
                continue
            pg = int(table[b, slot // page])
            if not 0 <= pg < k_cache.shape[0]:
                continue
            kc[pg, :, slot % page] = y[b, :, n]
            kb[pg, :, slot % page] = bound[b, :, n]
            vc[pg, :, slot % page] = v[b, :, n].double()
    return kc, kb, vc


def paged(q, k_cache, v_cache, table, lens, q_lens, prefix, prefix_len, scale, mask):
    """(o, bound, lse, bound), float64."""
    B, Hq, Nq, d = q.shape
    Hk, page = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hk
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)

    def rows(cache, pages, n):
        out = torch.zeros(Hk, n, d, dtype=torch.float64)
        for j in range(n):
            pg = int(pages[j // page])
            if 0 <= pg < cache.shape[0]:
                out[:, j] = cache[pg, :, j % page].double()
        return out

    kp, vp = (rows(c, prefix, prefix_len) for c in (k_cache, v_cache))
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        m = Nq if q_lens is None else max(0, min(Nq, int(q_lens[b])))
        k = torch.cat([kp, rows(k_cache, table[b], n)], 1)
        v = torch.cat([vp, rows(v_cache, table[b], n)], 1)
        total = prefix_len + n
        for i in range(m):
            seen = max(0, min(total, total - m + i + 1)) if mask == "causal_br" else total
            if seen == 0:
                continue
            for hk in range(Hk):
                qq = q[b, hk * G:(hk + 1) * G, i].double()
                kk, vv = k[hk, :seen], v[hk, :seen]
                s = scale * (qq @ kk.T)
                err = (d + 2) * T * scale * (qq.abs() @ kk.abs().T).amax(-1)
                p = torch.softmax(s, -1)
                hs = slice(hk * G, (hk + 1) * G)
                o[b, hs, i] = p @ vv
                ob[b, hs, i] = U * (p @ vv).abs() + (U + 2 * err + 2.0 ** -21)[:, None] * (p @ vv.abs())
                lse[b, hs, i] = torch.logsumexp(s, -1)
                lb[b, hs, i] = err + 2.0 ** -20 * (1 + lse[b, hs, i].abs())
    return o, ob, lse, lb


def check(name, got, ref, bound):
    got = got.detach().double().cpu()
    same = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), same), f"{name}: infinities or NaN in the wrong places"
    assert torch.equal(got[~same], ref[~same]), f"{name}: infinities differ"
    err = (got - ref).abs()[same]
    bad = err > bound[same]
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} out of bound, worst "
                           f"{float((err / bound[same].clamp(min=1e-300)).max()):.2f}")
