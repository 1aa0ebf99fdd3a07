"""GPU: attention over a paged cache with a shared prefix against its definition in
64 bits (bounds in cache_oracle), and a serving step of the cache operators together."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import cache_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from exact_attention_69_gb300 import build
    build.build()
    import exact_attention_69_gb300 as E
    return E


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


class Problem:
    """Inputs on the CPU: shuffled pages, NaN in every slot that no sequence holds, unused
    table entries that name no page."""

    def __init__(self, Hq, Hk, d, Nq, P, lens, page, q_lens=None, seed=0, scale_q=1.0):
        B = len(lens)
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        first = -(-P // page)
        self.n_pages = first + sum(need) + 1
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.prefix = torch.tensor(order[:first], dtype=torch.int32) if P else None
        self.table = torch.full((B, max(1, max(need))), 1 << 30, dtype=torch.int32)
        self.table[:, 1::2] = -7
        self.k, self.v = (rnd(seed + i, self.n_pages, Hk, page, d) for i in (1, 2))
        used = torch.zeros(self.n_pages, page, dtype=torch.bool)
        at = first
        for j in range(P):
            used[order[j // page], j % page] = True
        for b in range(B):
            ids = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
            for j in range(lens[b]):
                used[ids[j // page], j % page] = True
        for c in (self.k, self.v):
            c.masked_fill_(~used[:, None, :, None], float("nan"))
        self.q = rnd(seed + 3, B, Hq, Nq, d, scale=scale_q)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.q_lens = torch.tensor(q_lens, dtype=torch.int32) if q_lens is not None else None
        self.P, self.d = P, d

    def cuda(self):
        cu = lambda t: None if t is None else t.cuda()  # noqa: E731
        return [cu(t) for t in (self.q, self.k, self.v, self.table, self.lens, self.q_lens, self.prefix)]

    def want(self, mask="causal_br", lens=None):
        k, v = (c.nan_to_num(0.0) for c in (self.k, self.v))
        return O.paged(self.q, k, v, self.table, self.lens if lens is None else lens, self.q_lens, self.prefix, self.P,
                       1 / math.sqrt(self.d), mask)

    def run(self, E, mask="causal_br", **kw):
        q, k, v, table, lens, q_lens, prefix = self.cuda()
        return E.attn_paged(q, k, v, table, lens, q_lens=q_lens, prefix_table=prefix, prefix_len=self.P, mask=mask, **kw)

    def check(self, E, mask="causal_br", **kw):
        o, lse = self.run(E, mask, **kw)
        torch.cuda.synchronize()
        code, detail = E.device_status()
        assert code == 0, detail
        ro, bo, rl, bl = self.want(mask)
        O.check("o", o, ro, bo)
        O.check("lse", lse, rl, bl)


# Hq, Hk, d, Nq, P, lens, page, q_lens
CASES = [
    # one token: no prefix, one tile, cut nowhere
    (1, 1, 64, 1, 0, [1], 16, None),
    (4, 1, 128, 1, 0, [17], 16, None),
    (2, 2, 32, 1, 0, [128, 129, 0, 127], 32, None),
    # a prefix alone, and with own keys around the tile's and the page's ends
    (4, 2, 64, 1, 1, [0, 0], 16, None),
    (4, 2, 64, 1, 127, [1, 16], 16, None),
    (4, 2, 128, 1, 128, [15, 300, 0], 64, None),
    (8, 1, 32, 1, 129, [33, 200], 128, None),
    (7, 1, 128, 1, 1021, [511, 1, 0, 64], 32, None),
    (4, 4, 64, 1, 513, [130, 2], 256, None),
    # several tokens, their rows over one, two and more query tiles
    (6, 2, 64, 5, 40, [5, 200, 129], 16, None),
    (6, 2, 64, 5, 0, [5, 3, 0], 16, [5, 5, 2]),
    (3, 1, 128, 50, 260, [50, 333], 64, None),
    (3, 1, 64, 90, 260, [90, 133], 64, [90, 17]),
    (2, 2, 32, 300, 70, [300, 411], 32, None),
    (2, 1, 128, 150, 0, [150, 700, 20], 128, [150, 149, 20]),
    # more prefix rows than one task holds
    (8, 1, 64, 1, 300, [3] * 40, 16, None),
    (5, 5, 32, 9, 140, [9 + 3 * i for i in range(31)], 16, None),
    (16, 1, 128, 1, 130, [i % 4 for i in range(20)], 16, None),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_parity(E, case):
    Hq, Hk, d, Nq, P, lens, page, q_lens = case
    Problem(Hq, Hk, d, Nq, P, lens, page, q_lens, seed=100).check(E)


@pytest.mark.parametrize("mask", ["none", "causal_br"])
@pytest.mark.parametrize("ctas", [1, 2, 5, 37])
@pytest.mark.parametrize("case", [CASES[7], CASES[11], CASES[14], CASES[15]], ids=str)
def test_cuts(E, case, ctas, mask):
    """The same problem over other numbers of CTAs: tasks whole, cut in two, cut often."""
    Hq, Hk, d, Nq, P, lens, page, q_lens = case
    Problem(Hq, Hk, d, Nq, P, lens, page, q_lens, seed=200).check(E, mask, num_ctas=ctas)


@pytest.mark.parametrize("mask", ["none", "causal_br"])
@pytest.mark.parametrize("case", [c for c in CASES if c[4] > 0], ids=str)
def test_prefix_tasks(E, case, mask):
    """Few CTAs, where going over the prefix once for the batch pays earliest."""
    Hq, Hk, d, Nq, P, lens, page, q_lens = case
    Problem(Hq, Hk, d, Nq, P, lens, page, q_lens, seed=400).check(E, mask, num_ctas=2)


@pytest.mark.parametrize("case", [
    # prefix rows in boxes of several sequences, gathered, in one and in two query tiles
    (8, 2, 64, 1, 600, [(7 * i) % 90 for i in range(100)], 16, None),
    (4, 2, 32, 4, 700, [(11 * i) % 70 for i in range(90)], 32, [1 + i % 4 for i in range(90)]),
    (6, 2, 128, 5, 500, [(13 * i) % 60 for i in range(120)], 16, None),
    (4, 4, 64, 8, 1500, [(5 * i) % 40 for i in range(16)], 64, None),
    # rows of many parts each: more than eight, and more than one warp's share
    (4, 1, 128, 1, 6000, [3000, 2500], 64, None),
    (4, 2, 64, 4, 7000, [50, 4000, 0], 16, None),
    (2, 1, 32, 2, 17000, [100], 128, None),
    (1, 1, 64, 1, 0, [20000], 256, None),
], ids=str)
def test_shared_prefixes_and_many_parts(E, case):
    Hq, Hk, d, Nq, P, lens, page, q_lens = case
    Problem(Hq, Hk, d, Nq, P, lens, page, q_lens, seed=450).check(E)


def test_rising_maxima(E):
    """Scores that grow along the keys (the running maximum is raised tile after tile) and
    parts whose maxima are far apart."""
    p = Problem(4, 1, 64, 1, 700, [650, 10], 32, seed=300, scale_q=4.0)
    ramp = torch.linspace(0.1, 6.0, 22)
    for j, pg in enumerate(p.prefix.tolist()):
        p.k[pg] *= ramp[j]
    for j, pg in enumerate(p.table[0].tolist()):
        p.k[pg] *= ramp[21 - j]
    for ctas in (0, 3):
        p.check(E, num_ctas=ctas)


def test_layouts(E):
    """Heads-last queries and outputs, [page, slot, head, d] caches, a wider table."""
    p = Problem(6, 3, 64, 4, 100, [77, 210], 32, seed=400)
    q, k, v, table, lens, _, prefix = p.cuda()
    qh = q.transpose(1, 2).contiguous().transpose(1, 2)
    kn, vn = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    wide = torch.full((2, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out = torch.empty(2, 4, 6, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    o = E.attn_paged(qh, kn, vn, wide, lens, prefix_table=prefix, prefix_len=100, out=out, return_lse=False)
    o2, _ = E.attn_paged(q, k, v, table, lens, prefix_table=prefix, prefix_len=100)
    assert o.data_ptr() == out.data_ptr() and torch.equal(o, o2)
    ro, bo, _, _ = p.want()
    O.check("o", o, ro, bo)


def test_lengths_beyond_the_table_are_cut(E):
    p = Problem(2, 1, 32, 1, 0, [48, 20], 16, seed=500)
    q, k, v, table, _, _, _ = p.cuda()
    big = torch.tensor([1 << 30, -5], dtype=torch.int32)
    o, lse = E.attn_paged(q, k, v, table, big.cuda())
    ro, bo, rl, bl = p.want(lens=big)
    O.check("o", o, ro, bo)
    O.check("lse", lse, rl, bl)
    assert float(o[1].abs().max()) == 0.0


def test_pages_that_the_cache_has_not(E):
    """Entries that name no page read as zeros: scores and values 0, nothing outside."""
    p = Problem(2, 1, 64, 1, 0, [64], 16, seed=600)
    p.table[0, 1], p.table[0, 3] = p.n_pages, -1
    p.check(E)


def test_same_bits_twice_and_two_streams(E):
    """No atomics: equal bits; two calls at once on two streams have their own scratch."""
    a = Problem(8, 2, 128, 1, 900, [100, 700, 33], 16, seed=700)
    b = Problem(4, 4, 64, 3, 300, [10, 900], 64, seed=701)
    ra, rb = a.run(E), b.run(E)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        xa, xb = a.run(E, stream=s1), b.run(E, stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(xa + xb, ra + rb))


def test_graph_follows_the_lengths(E):
    p = Problem(4, 2, 64, 1, 200, [300, 300, 300], 32, seed=800)
    q, k, v, table, lens, _, prefix = p.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = E.attn_paged(q, k, v, table, lens, prefix_table=prefix, prefix_len=200)
    for now in ([300, 300, 300], [1, 128, 257], [0, 0, 5]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        ro, bo, rl, bl = p.want(lens=now)
        O.check("o", o, ro, bo)
        O.check("lse", lse, rl, bl)


def test_many_sequences(E):
    """More sequences than threads of a block, most of them short or empty."""
    lens = [(7 * i) % 23 if i % 3 else 0 for i in range(900)]
    Problem(2, 1, 32, 1, 50, lens, 16, seed=900).check(E)


@pytest.mark.parametrize("seed", range(16))
def test_random_problems(E, seed):
    """Sizes drawn at random: groups of heads, lengths, pages, cuts, padding."""
    r = random.Random(seed)
    Hk, G, d = r.choice([1, 2, 3]), r.choice([1, 2, 4, 5, 8, 16]), r.choice([32, 64, 128])
    Nq = r.choice([1, 1, 2, r.randint(3, 20), r.randint(60, 140)])
    B = r.randint(1, 9 if Nq < 21 else 3)
    page = r.choice([16, 32, 64, 128, 512])
    q_lens = [r.randint(0, Nq) for _ in range(B)] if r.random() < 0.4 else None
    lens = [max(r.choice([0, 1, r.randint(2, 600)]), q_lens[b] if q_lens else Nq) if r.random() < 0.8 else r.randint(0, 40)
            for b in range(B)]
    P = r.choice([0, 0, r.randint(1, 130), r.randint(200, 1500)])
    Problem(Hk * G, Hk, d, Nq, P, lens, page, q_lens, seed=2000 + 10 * seed).check(
        E, r.choice(["none", "causal_br"]), num_ctas=r.choice([0, 0, r.randint(1, 60)]))


def test_offsets_beyond_32_bits(E):
    """Caches of more than 2^31 elements: their last pages are written and read."""
    Hk, page, d, n_pages = 8, 64, 128, 33000
    kc, vc = (torch.empty(n_pages, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    table = torch.tensor([[n_pages - 1, 3], [n_pages - 2, n_pages - 3]], dtype=torch.int32)
    small = {int(p): i for i, p in enumerate(sorted(set(table.flatten().tolist())))}
    k, v = rnd(31, 2, Hk, 100, d), rnd(32, 2, Hk, 100, d)
    E.kv_append(k.cuda(), v.cuda(), kc, vc, table.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"))
    q = rnd(33, 2, Hk, 1, d)
    o, lse = E.attn_paged(q.cuda(), kc, vc, table.cuda(), torch.tensor([100, 77], dtype=torch.int32, device="cuda"))
    ks, vs = (torch.stack([c[p].cpu() for p in small]).nan_to_num(0.0) for c in (kc, vc))
    for b in range(2):
        for j in range(100):
            pg = small[int(table[b, j // page])]
            assert torch.equal(ks[pg, :, j % page], k[b, :, j]) and torch.equal(vs[pg, :, j % page], v[b, :, j])
    remap = torch.tensor([[small[int(p)] for p in row] for row in table], dtype=torch.int32)
    ro, bo, rl, bl = O.paged(q, ks, vs, remap, [100, 77], None, None, 0, 1 / math.sqrt(d), "causal_br")
    O.check("o", o, ro, bo)
    O.check("lse", lse, rl, bl)


def test_keys_and_values_in_one_tensor(E):
    """Caches that are views of one [page, 2, head, slot, d] tensor."""
    p = Problem(4, 2, 64, 1, 90, [130, 40], 32, seed=1300)
    kv = torch.stack([p.k, p.v], dim=1).cuda()
    q, _, _, table, lens, _, prefix = p.cuda()
    o, lse = E.attn_paged(q, kv[:, 0], kv[:, 1], table, lens, prefix_table=prefix, prefix_len=90)
    ro, bo, rl, bl = p.want()
    O.check("o", o, ro, bo)
    O.check("lse", lse, rl, bl)


def test_first_calls_captured():
    """In a new process the first call of each operator may be a captured one."""
    code = """
import torch, exact_attention_69_gb300 as E
t = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")
k, kc, vc, q = t(2, 2, 3, 64), t(4, 2, 16, 64), t(4, 2, 16, 64), t(2, 4, 3, 64)
table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
f, w = E.rope_freqs(64), torch.ones(64, device="cuda")
lens = starts + 3
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qr = E.kv_append(k, k, kc, vc, table, starts, inv_freq=f, eps=1e-6, q=q)
    o, lse = E.attn_paged(qr, kc, vc, table, lens)
    a, b = E.qk_norm_rope_fwd(q, k, w, w, inv_freq=f)
    grads = E.qk_norm_rope_bwd(q, k, a, b, w, w, inv_freq=f)
g.replay()
torch.cuda.synchronize()
assert E.device_status()[0] == 0 and bool(torch.isfinite(o).all()) and bool((o == 1).all())
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_refusals(E):
    """What the host can see is refused before anything runs."""
    p = Problem(4, 2, 64, 2, 20, [30, 9], 16, seed=1400)
    q, k, v, table, lens, _, prefix = p.cuda()
    call = lambda **kw: E.attn_paged(**{**dict(q=q, k_cache=k, v_cache=v, block_table=table, kv_lens=lens,  # noqa: E731
                                               prefix_table=prefix, prefix_len=20), **kw})
    for bad in (dict(q=q.float()), dict(kv_lens=lens.long()), dict(kv_lens=lens[:1]), dict(block_table=table[:1]),
                dict(v_cache=v[:, :1]), dict(k_cache=k[:, :, :, :32]), dict(mask="causal"), dict(kv_lens=lens.cpu()),
                dict(out=q[:1]), dict(lse=torch.empty(2, 4, 2, device="cuda", dtype=torch.float64)),
                dict(q=q.transpose(2, 3)), dict(q_lens=lens.float())):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    for bad in (dict(prefix_len=-1), dict(prefix_len=33), dict(prefix_table=None), dict(scale=0.0), dict(scale=float("nan")),
                dict(q=q[:, :3].contiguous()), dict(q=q.new_empty(0, 4, 2, 64), block_table=table[:0], kv_lens=lens[:0])):
        with pytest.raises(E.AttnError):
            call(**bad)
    call()


def test_timeout_is_reported(E):
    """A withheld K tile: the bounded wait runs out and the status says so; the next call
    is right."""
    p = Problem(4, 1, 64, 1, 0, [700], 16, seed=1000)
    p.run(E, num_ctas=1, timeout_ns=20_000_000, inject=1)
    torch.cuda.synchronize()
    code, detail = E.device_status()
    assert code == 5 and detail[0] == 5
    p.check(E)


def test_timeout_before_the_task_table_is_written(E, monkeypatch):
    """One CTA stops at its second tile, with tasks that it never noted for the join: a
    workspace full of large numbers must not send the join anywhere else, with and
    without a batched prefix, and the next call is right."""
    empty = torch.empty

    def full(*a, **kw):
        t = empty(*a, **kw)
        return t.fill_(0x7F) if t.dtype == torch.uint8 else t

    for P in (0, 2000):
        p = Problem(4, 1, 64, 1, P, [700] * 24, 16, seed=1010)
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", full)
            p.run(E, num_ctas=1, timeout_ns=20_000_000, inject=1)
        torch.cuda.synchronize()
        assert E.device_status()[0] == 5
        p.check(E)


def test_options_by_value(E):
    """Options given as tensors are read at each call, not when their combination was first seen."""
    p = Problem(4, 2, 64, 1, 60, [40, 7], 16, seed=1020)
    n = torch.tensor(30)
    q, k, v, table, lens, _, prefix = p.cuda()
    E.attn_paged(q, k, v, table, lens, prefix_table=prefix, prefix_len=n)
    n.fill_(60)
    o, lse = E.attn_paged(q, k, v, table, lens, prefix_table=prefix, prefix_len=n)
    ro, bo, rl, bl = p.want()
    O.check("o", o, ro, bo)
    O.check("lse", lse, rl, bl)


def test_serving_steps(E):
    """Prompt chunk and decoding steps over one cache: norm, rotation, append and attention
    as a server runs them, against the same steps in 64 bits."""
    B, Hq, Hk, d, page, P = 3, 6, 2, 64, 16, 37
    freqs = E.rope_freqs(d)
    wq, wk = (1 + 0.2 * rnd(i, d).float() for i in (1, 2))
    p = Problem(Hq, Hk, d, 1, P, [60, 60, 60], page, seed=1100)
    kc, vc = p.k.cuda(), p.v.cuda()
    table, prefix = p.table.cuda(), p.prefix.cuda()
    ok, ov = p.k.nan_to_num(0.0).double(), p.v.nan_to_num(0.0).double()
    held = torch.zeros(B, dtype=torch.int32)
    bound = torch.zeros_like(ok)
    for step, (N, counts) in enumerate([(20, [20, 7, 13]), (1, None), (1, None), (4, [4, 1, 3])]):
        x = rnd(1200 + step, B, N, Hq + 2 * Hk, d).cuda()
        q, k, v = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2), x[:, :, Hq + Hk:].transpose(1, 2)
        new = torch.tensor(counts if counts else [N] * B, dtype=torch.int32)
        cnt = new.cuda() if counts else None
        start = held.cuda()
        qr = E.kv_append(k, v, kc, vc, table, start, counts=cnt, position_offset=P, inv_freq=freqs, eps=1e-6,
                         k_weight=wk.cuda(), q=q, q_weight=wq.cuda())
        o, lse = E.attn_paged(qr, kc, vc, table, start + new.cuda(), q_lens=cnt, prefix_table=prefix, prefix_len=P)
        pos = P + held[:, None] + torch.arange(N)
        ok, kb, ov = O.append(k.cpu(), v.cpu(), ok, ov, p.table, held, cnt.cpu() if counts else None, pos,
                              freqs.cpu(), False, 1e-6, wk)
        bound += kb
        held = held + new
        for b in range(B):
            for j in range(int(held[b])):
                pg = int(p.table[b, j // page])
                err = (kc[pg, :, j % page].cpu().double() - ok[pg, :, j % page]).abs()
                assert bool((err <= bound[pg, :, j % page]).all())
                assert torch.equal(vc[pg, :, j % page].cpu().double(), ov[pg, :, j % page])
        # attention is held to the keys that the cache has
        k64, v64 = kc.cpu().double().nan_to_num(0.0), vc.cpu().double().nan_to_num(0.0)
        ro, bo, rl, bl = O.paged(qr.cpu(), k64, v64, p.table, held, cnt.cpu() if counts else None, p.prefix, P,
                                 1 / math.sqrt(d), "causal_br")
        O.check("o", o, ro, bo)
        O.check("lse", lse, rl, bl)
        O.check("q", qr, *O.norm_rope(q.cpu(), wq, pos, freqs.cpu(), False, 1e-6))
    torch.cuda.synchronize()
    assert E.device_status()[0] == 0
