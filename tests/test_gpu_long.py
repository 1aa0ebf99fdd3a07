"""GPU: the long-cache operators against their definitions in 64 bits (bounds in
long_oracle), and a server's steps that use them together."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import long_oracle as O
from tests.cache_oracle import check

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def done(E):
    """Nothing that a device wait ran out for."""
    torch.cuda.synchronize()
    code, detail = E.device_status()
    assert code == 0, detail


# by the library's rule, and with tiles of 128 rows whatever the sizes
FORMS = pytest.mark.parametrize("full", [None, True], ids=["rule", "full"])


class Problem:
    """Inputs on the CPU: shuffled pages, NaN in every slot that no sequence holds, unused
    table entries that name no page."""

    def __init__(self, Hq, Hk, d, Nq, lens, page, q_lens=None, seed=0, spare=1, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(1, width or 0, max(need))), 1 << 30, dtype=torch.int32)
        self.table[:, 1::2] = -7
        self.k, self.v = (rnd(seed + i, self.n_pages, Hk, page, d) for i in (1, 2))
        # pages differ, so that scores do
        self.k += rnd(seed + 5, self.n_pages, Hk, 1, d)
        self.w = torch.rand(self.n_pages, Hk, page, generator=g) * 4
        used = torch.zeros(self.n_pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(lens):
            ids = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = ints(ids)
            for j in range(n):
                used[ids[j // page], j % page] = True
        self.spare = ints(order[at:])
        for c in (self.k, self.v):
            c.masked_fill_(~used[:, None, :, None], float("nan"))
        self.w.masked_fill_(~used[:, None], float("nan"))
        self.q = rnd(seed + 3, len(lens), Hq, Nq, d)
        self.lens, self.q_lens = ints(lens), None if q_lens is None else ints(q_lens)
        self.page, self.d, self.Hk, self.Nq, self.G = page, d, Hk, Nq, Hq // Hk
        self.scale = 1 / math.sqrt(d)

    def k0(self):
        return self.k.nan_to_num(0.0)

    def lists(self, n, seed=0):
        """Lists of any order, with entries that name nothing and some twice."""
        g = torch.Generator().manual_seed(seed)
        W = self.table.shape[1]
        return torch.randint(-2, W + 3, (len(self.lens), self.Hk, self.Nq, n), generator=g, dtype=torch.int32)

    def run_blocks(self, E, lists, mask="causal_br", **kw):
        return E.attn_blocks(self.q.cuda(), self.k.cuda(), self.v.cuda(), self.table.cuda(), self.lens.cuda(), lists.cuda(),
                             q_lens=None if self.q_lens is None else self.q_lens.cuda(), mask=mask, **kw)

    def check_blocks(self, E, lists, mask="causal_br", **kw):
        o, lse = self.run_blocks(E, lists, mask, **kw)
        done(E)
        ro, bo, rl, bl = O.blocks(self.q, self.k0(), self.v.nan_to_num(0.0), self.table, self.lens, lists, self.q_lens,
                                  self.scale, mask)
        check("o", o, ro, bo)
        check("lse", lse, rl, bl)

    def check_scores(self, E, mask="causal_br", **kw):
        bnd = torch.zeros(self.n_pages, self.Hk, 2, self.d, dtype=torch.bfloat16)
        got = bnd.cuda()
        E.kv_bounds(self.k.cuda(), got, self.table.cuda(), self.lens.cuda())
        want = O.bounds(self.k, bnd, self.table, self.lens, None)
        assert torch.equal(got.cpu(), want)
        s = E.block_scores(self.q.cuda(), got, self.table.cuda(), self.lens.cuda(), page_size=self.page,
                           q_lens=None if self.q_lens is None else self.q_lens.cuda(), mask=mask, **kw)
        done(E)
        check("scores", s, *O.scores(self.q, want, self.table, self.lens, self.q_lens, self.page, self.scale, mask))
        return s

    def check_weights(self, E, mask="causal_br", decay=1.0, lse=None, **kw):
        if lse is None:
            k, g = self.k0(), torch.Generator().manual_seed(9)
            lse = 2 + torch.rand(self.q.shape[:3], generator=g)
        got = self.w.cuda()
        E.kv_weights(self.q.cuda(), self.k.cuda(), self.table.cuda(), self.lens.cuda(), lse.cuda(), got,
                     q_lens=None if self.q_lens is None else self.q_lens.cuda(), mask=mask, decay=decay, **kw)
        done(E)
        ref, err = O.weights(self.q, self.k0(), self.table, self.lens, lse, self.w, self.q_lens, self.scale, mask, decay)
        nan = ref.isnan()
        assert torch.equal(got.cpu().isnan(), nan)
        check("weights", got.cpu().nan_to_num(0.0), ref.nan_to_num(0.0), err)


# Hq, Hk, d, Nq, lens, page, q_lens
CASES = [
    (1, 1, 64, 1, [1], 16, None),
    (4, 1, 128, 1, [17, 0, 16], 16, None),
    (2, 2, 32, 1, [128, 129, 0, 127], 32, None),
    (8, 2, 64, 1, [1000, 3], 16, None),
    (7, 1, 128, 1, [511, 1, 0, 64], 64, None),
    (9, 1, 64, 1, [300], 128, None),
    (32, 2, 32, 1, [260, 77], 16, None),
    (48, 1, 128, 1, [200], 32, None),
    (6, 2, 64, 5, [5, 200, 129], 16, None),
    (6, 2, 64, 5, [5, 3, 0], 16, [5, 5, 2]),
    (3, 1, 128, 50, [50, 333], 64, None),
    (3, 1, 64, 90, [90, 133], 64, [90, 17]),
    (2, 2, 32, 140, [300, 411], 32, None),
    (4, 1, 64, 33, [700, 40], 16, [0, 33]),
    (10, 2, 128, 7, [600], 256, None),
    (1, 1, 32, 20, [1900], 16, None),
]


@FORMS
@pytest.mark.parametrize("mask", ["causal_br", "none"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_scores(E, case, mask, full):
    Hq, Hk, d, Nq, lens, page, q_lens = case
    Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=100).check_scores(E, mask, full_tiles=full)


@FORMS
@pytest.mark.parametrize("mask", ["causal_br", "none"])
@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_blocks(E, case, n, mask, full):
    Hq, Hk, d, Nq, lens, page, q_lens = case
    p = Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=200)
    p.check_blocks(E, p.lists(n, seed=n), mask, full_tiles=full)


@FORMS
@pytest.mark.parametrize("mask", ["causal_br", "none"])
@pytest.mark.parametrize("decay", [0.0, 1.0, 0.5])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_weights(E, case, decay, mask, full):
    Hq, Hk, d, Nq, lens, page, q_lens = case
    Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=300).check_weights(E, mask, decay, full_tiles=full)


@pytest.mark.parametrize("n_new", [0, 1, 2, 16, 17, 33, 1000])
def test_bounds_of_new_tokens(E, n_new):
    """Only pages that hold a new token are written, each from all of its live slots."""
    p = Problem(2, 2, 64, 1, [1, 16, 17, 0, 250, 33], 16, seed=400)
    old = rnd(401, p.n_pages, 2, 2, 64)
    got = old.cuda()
    E.kv_bounds(p.k.cuda(), got, p.table.cuda(), p.lens.cuda(), n_new=n_new)
    assert torch.equal(got.cpu(), O.bounds(p.k, old, p.table, p.lens, n_new))


def test_bounds_of_nan_and_infinities(E):
    p = Problem(2, 1, 32, 1, [48, 20], 16, seed=410)
    ids = p.table[0].tolist()
    p.k[ids[0], 0, 3, 5], p.k[ids[1], 0, 0, 6], p.k[ids[1], 0, 1, 7] = float("nan"), float("inf"), -float("inf")
    b = torch.zeros(p.n_pages, 1, 2, 32, dtype=torch.bfloat16, device="cuda")
    E.kv_bounds(p.k.cuda(), b, p.table.cuda(), p.lens.cuda())
    assert torch.equal(b.cpu().nan_to_num(9.0), O.bounds(p.k, b.cpu() * 0, p.table, p.lens, None).nan_to_num(9.0))
    assert bool(b[ids[0], 0, :, 5].isnan().all())
    s = E.block_scores(p.q.cuda(), b, p.table.cuda(), p.lens.cuda(), page_size=16)
    assert bool(s[0, 0, 0, 0].isnan()) and not bool(s[0, 0, 0, 2].isnan())
    # NaN is selected before everything else
    took = E.block_select(torch.tensor([[[[1.0, 9.0, float("nan"), 3.0]]]]).cuda(), ints([64]).cuda(), 2, page_size=16,
                          first=0, last=0)
    assert took.tolist() == [[[[1, 2]]]]


@FORMS
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 11, 16, 24, 70])
def test_scores_of_head_groups(E, G, full):
    Problem(2 * G, 2, 32, 9, [100, 300], 16, seed=420 + G).check_scores(E, full_tiles=full)


def test_scores_of_many_pages_and_tokens(E):
    """Several tiles of pages and several runs of tokens."""
    Problem(4, 1, 64, 200, [16 * 300, 16 * 140], 16, [200, 77], seed=430).check_scores(E)
    Problem(6, 2, 128, 90, [16 * 200 + 5], 16, seed=431).check_scores(E, "none")


@FORMS
def test_scores_of_negative_queries(E, full):
    """Every head of a group scores below zero: padding must not win."""
    p = Problem(3, 1, 64, 2, [200], 16, seed=440)
    p.q, p.k = -p.q.abs() - 1, p.k.abs() + 1
    s = p.check_scores(E, full_tiles=full)
    assert bool((s[s > -math.inf] < 0).all())


# widths around the sizes of the teams that share a row
@pytest.mark.parametrize("W", [1, 2, 5, 127, 128, 129, 511, 512, 513, 1024, 1025, 4096, 4097, 16384, 16385, 40001])
def test_select(E, W):
    g = torch.Generator().manual_seed(W)
    B, Hk, Nq, page = 2, 2, 3, 16
    lens, q_lens = ints([W * page, max(1, W * page - W * 5)]), ints([3, 2])
    s = torch.randn(B, Hk, Nq, W, generator=g)
    s[0, 0] = (s[0, 0] * 2).round() / 2          # ties
    s[1, 1, 0] = 0.25
    s[1, 1, 0, ::3] = -0.0
    s[1, 1, 1, ::2] = 0.0
    s[0, 1, 0, W // 2] = float("nan")
    s[0, 1, 1, W // 3] = math.inf
    s[0, 1, 2] = -math.inf
    s[0, 1, 2, W // 2:] = -3e38
    for n, first, last in ((1, 0, 0), (4, 1, 2), (33, 0, 5), (W, 1, 0) if W > 1 else (7, 1, 2), (max(1, W - 1), 0, 0)):
        for mask in ("causal_br", "none"):
            got = E.block_select(s.cuda(), lens.cuda(), n, page_size=page, q_lens=q_lens.cuda(), first=first, last=last,
                                 mask=mask)
            assert torch.equal(got.cpu(), O.select(s, lens, q_lens, n, page, first, last, mask)), (n, first, last, mask)


def test_select_ignores_what_a_query_does_not_see(E):
    """Scores behind the last visible page may hold anything; padded queries select nothing."""
    s = torch.full((1, 1, 4, 50), float("nan"))
    s[..., :3] = torch.tensor([3.0, 1.0, 2.0])
    got = E.block_select(s.cuda(), ints([3 * 32]).cuda(), 2, page_size=32, q_lens=ints([2]).cuda(), first=0, last=0)
    assert got.tolist() == [[[[0, 2], [0, 2], [-1, -1], [-1, -1]]]]


def test_blocks_equal_paged_where_every_page_is_selected(E):
    """The same attention as attn_paged's if the lists name all pages, in any order."""
    for Hq, Hk, d, Nq, lens, page, q_lens in CASES[3:14]:
        p = Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=500)
        W = p.table.shape[1]
        lists = torch.stack([torch.randperm(W) for _ in range(len(lens) * Hk * Nq)]).int().reshape(len(lens), Hk, Nq, W)
        p.check_blocks(E, lists)
        o, lse = p.run_blocks(E, lists)
        o2, lse2 = E.attn_paged(p.q.cuda(), p.k.cuda(), p.v.cuda(), p.table.cuda(), p.lens.cuda(),
                                q_lens=None if p.q_lens is None else p.q_lens.cuda())
        same = torch.isfinite(lse2)
        assert torch.equal(same, torch.isfinite(lse)) and float((lse - lse2)[same].abs().max()) < 2.0 ** -17
        assert float((o.float() - o2.float()).abs().max()) < 0.05


@FORMS
def test_blocks_of_wide_tables(E, full):
    """More pages than the bits in shared memory cover at a time."""
    p = Problem(4, 2, 32, 1, [16 * 2500 + 3, 40], 16, seed=520)
    p.check_blocks(E, p.lists(64, seed=1), full_tiles=full)
    p = Problem(2, 1, 32, 6, [16 * 3300, 100], 16, seed=521)
    p.check_blocks(E, p.lists(30, seed=2), full_tiles=full)


@FORMS
@pytest.mark.parametrize("n", [1, 2, 31, 40, 127, 128, 129, 200])
@pytest.mark.parametrize("Hq,Hk,d,lens,page", [
    (4, 2, 64, [16 * 90 + 5, 1, 0, 300], 16),
    (3, 1, 128, [64 * 150 + 63], 64),
    (10, 1, 32, [32 * 20, 32 * 64 + 1], 32),
], ids=str)
def test_blocks_of_one_query(E, Hq, Hk, d, lens, page, n, full):
    """Lists shorter and longer than what a block takes at once, many entries twice or more."""
    p = Problem(Hq, Hk, d, 1, lens, page, seed=540 + n)
    p.check_blocks(E, p.lists(n, seed=n), full_tiles=full)


@FORMS
@pytest.mark.parametrize("Hq,Hk,d,Nq,lens,page,n", [
    (4, 1, 32, 20, [16 * 2600 + 9, 16 * 1025], 16, 5),    # 20 queries a tile
    (2, 1, 64, 70, [16 * 1100 + 1, 16 * 511 + 3], 16, 4),  # up to 64
    (1, 1, 32, 150, [16 * 800 + 2, 16 * 257], 16, 3),     # up to 128
], ids=str)
@pytest.mark.parametrize("spread", ["anywhere", "ends", "edges", "last", "none"])
def test_blocks_far_apart(E, Hq, Hk, d, Nq, lens, page, n, spread, full):
    """Pages at random, at the two ends, next to multiples of 256, the last alone, none."""
    p = Problem(Hq, Hk, d, Nq, lens, page, seed=545)
    W = p.table.shape[1]
    lists = p.lists(n, seed=7)
    last = ((p.lens - 1) // page)[:, None, None, None].expand_as(lists)
    if spread == "ends":
        lists = torch.where(lists % 2 == 0, lists % 5, last - lists % 5)
    elif spread == "edges":
        lists = lists // 256 * 256 + lists % 3 - 1
    elif spread == "last":
        lists = last.clone()
    elif spread == "none":
        lists = torch.where(lists % 2 == 0, -1, W + 5)
    p.check_blocks(E, lists.int().contiguous(), full_tiles=full)


# full tiles whose stages two, four or eight blocks share: 2, 4, 8 of lists of 8, 16 and 32
# stages (d = 32: four at most), windows of fewer stages than blocks, ragged counts, rows
# that select nothing, heads that do not divide a tile
@pytest.mark.parametrize("Hq,Hk,d,Nq,lens,page,q_lens,n", [
    (4, 2, 64, 3, [2000, 1, 0], 64, None, 8),
    (3, 1, 128, 50, [3000, 50], 64, [50, 17], 17),
    (8, 1, 128, 20, [64 * 70 + 1], 64, [13], 40),
    (2, 2, 32, 70, [900, 2000], 32, [70, 1], 70),
    (5, 1, 64, 33, [16 * 600 + 1, 16 * 70], 16, None, 130),
    (2, 1, 64, 130, [256 * 9 + 200], 256, None, 9),
    (6, 2, 128, 1, [512 * 6 + 5, 100], 512, None, 5),
    (7, 1, 32, 9, [16 * 2000 + 7], 16, None, 70),
], ids=str)
@pytest.mark.parametrize("mask", ["causal_br", "none"])
def test_blocks_shared_by_a_cluster(E, Hq, Hk, d, Nq, lens, page, q_lens, n, mask):
    p = Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=550)
    lists = p.lists(n, seed=5)
    lists[:, :, ::7] = -1
    p.check_blocks(E, lists, mask, full_tiles=True)
    same = p.run_blocks(E, lists, mask, full_tiles=True)
    again = p.run_blocks(E, lists, mask, full_tiles=True)
    assert all(torch.equal(x, y) for x, y in zip(same, again))
    # one page a query: most blocks of a cluster have nothing
    lists[..., 1:] = -1
    p.check_blocks(E, lists, mask, full_tiles=True)


def test_blocks_of_a_cluster_with_scores_that_are_not_finite(E):
    """A NaN or +inf score reaches its row from whichever block met it; rows of other queries,
    whose pages it is not on, keep their values."""
    p = Problem(2, 1, 64, 4, [64 * 32], 64, seed=555)
    want = torch.arange(32, dtype=torch.int32).expand(1, 1, 4, 32).contiguous()
    for bad in (float("nan"), float("inf")):
        for page in (0, 13, 31):
            k = p.k.clone()
            k[p.table[0, page], 0, 5] = bad if bad != bad else torch.sign(p.q[0, 0, 3].float()).bfloat16() * bad
            lists = want.clone()
            lists[0, 0, :3, page] = -1  # (queries 0 to 2 did not select it)
            o, lse = E.attn_blocks(p.q.cuda(), k.cuda(), p.v.cuda(), p.table.cuda(), p.lens.cuda(), lists.cuda(),
                                   mask="none", full_tiles=True)
            done(E)
            assert bool(o[0, 0, 3].isnan().all()) and bool(lse[0, 0, 3].isnan())
            ro, bo, rl, bl = O.blocks(p.q, p.k0(), p.v.nan_to_num(0.0), p.table, p.lens, lists, None, p.scale, "none")
            check("o", o[:, :, :3], ro[:, :, :3], bo[:, :, :3])
            check("lse", lse[:, :, :3], rl[:, :, :3], bl[:, :, :3])


def test_clusters_of_calls_at_once(E):
    """Calls on several streams, also captured and replayed, whose blocks share tiles: the same bits."""
    ps = [Problem(4, 2, d, 90, [64 * 30, 64 * 12 + 5, 700], 64, seed=557 + d) for d in (32, 64, 128)]
    args = [tuple(x.cuda() for x in (p.q, p.k, p.v, p.table, p.lens, p.lists(24))) for p in ps]
    want = [E.attn_blocks(*a, full_tiles=True) for a in args]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = [E.attn_blocks(*a, full_tiles=True) for a in args for _ in range(2)]
    for _ in range(5):
        got = [[E.attn_blocks(*a, full_tiles=True, stream=s) for _ in range(3)] for a, s in zip(args, streams)]
        g.replay()
        torch.cuda.synchronize()
        for x, y in [(x, w) for w, runs in zip(want, got) for x in runs] + list(zip(held, [w for w in want for _ in range(2)])):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    done(E)


def test_timeouts_of_a_cluster_are_reported(E):
    p = Problem(4, 1, 64, 40, [64 * 40], 64, seed=556)
    lists = p.lists(32)
    p.run_blocks(E, lists, full_tiles=True, timeout_ns=20_000_000, inject=1)
    torch.cuda.synchronize()
    assert E.device_status()[0] != 0
    p.check_blocks(E, lists, full_tiles=True)


@pytest.mark.parametrize("Hq,Hk,d,Nq,lens,page,n", [
    (4, 2, 64, 1, [40, 3], 16, 4),
    (8, 2, 128, 20, [64 * 9 + 7, 30], 64, 3),
    (3, 1, 32, 50, [700], 32, 6),
    (2, 1, 64, 130, [64 * 40], 64, 33),
    (4, 1, 128, 500, [800], 64, 9),
], ids=str)
def test_blocks_with_weights_in_two_parts(E, Hq, Hk, d, Nq, lens, page, n):
    """What a caller who asks for the form for few rows gets at any size: the output's own
    rounding is nearly all of the error."""
    p = Problem(Hq, Hk, d, Nq, lens, page, seed=559)
    lists = p.lists(n, seed=8)
    o, _ = p.run_blocks(E, lists, full_tiles=False)
    done(E)
    check("o", o, *O.blocks_two_parts(p.q, p.k0(), p.v.nan_to_num(0.0), p.table, p.lens, lists, None, p.scale, "causal_br",
                                      n * page))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens", [[64 * 40], [64 * 6]], ids=["cluster", "few stages"])
def test_blocks_that_give_up_with_copies_on_their_way(E, d, lens):
    """The shortest limit, and values that come after it: a block gives up between a stage's S
    and its O, waits for what is in flight, reports it and leaves nothing behind for the next call."""
    p = Problem(4, 1, d, 40, lens, 64, seed=558)
    lists = p.lists(24, seed=6)
    for _ in range(2):
        p.run_blocks(E, lists, full_tiles=True, timeout_ns=1, inject=-1)
        torch.cuda.synchronize()
        code, detail = E.device_status()
        assert code == 5 and detail[0] == 5
        p.check_blocks(E, lists, full_tiles=True)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("pages", [1, 2, 3, 4, 7])
def test_blocks_whose_values_come_late(E, d, pages):
    """S = Q K^T runs a stage ahead of O += P V: a row that is through with its last stage's
    softmax waits for that stage's O although the one before is not done either."""
    p = Problem(8, 2, d, 40, [64 * pages, 64 * 20], 64, seed=560 + pages)
    lists = torch.arange(pages, dtype=torch.int32).expand(2, 2, 40, pages).contiguous()
    for mask in ("none", "causal_br"):
        p.check_blocks(E, lists, mask, full_tiles=True, inject=-1)
        late, on_time = p.run_blocks(E, lists, mask, full_tiles=True, inject=-1), p.run_blocks(E, lists, mask, full_tiles=True)
        assert all(torch.equal(x, y) for x, y in zip(late, on_time))


@pytest.mark.parametrize("Hq,Hk,d,Nq,lens,page,q_lens,n", [
    # enough rows for tiles of 128 by the rule: one query after another, heads that do not
    # divide a tile, pages smaller and larger than a stage, ragged counts, a short sequence
    (8, 2, 128, 1000, [1100], 64, None, 6),
    (3, 1, 64, 1300, [1300, 1500], 16, [1300, 1290], 9),
    (12, 4, 32, 700, [4000], 32, None, 5),
    (16, 1, 64, 500, [900], 128, [471], 4),
    (2, 2, 128, 1900, [1900, 2000], 256, [0, 1900], 3),
    (5, 1, 32, 1500, [3], 16, None, 2),
], ids=str)
def test_blocks_of_many_rows(E, Hq, Hk, d, Nq, lens, page, q_lens, n):
    p = Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=525)
    p.check_blocks(E, p.lists(n, seed=4))


@pytest.mark.parametrize("Hq,Hk,d,Nq,lens,page,q_lens,n", [
    (8, 2, 128, 400, [1100], 64, None, 6),
    (3, 1, 64, 300, [330, 1500], 16, [300, 290], 9),
    (16, 1, 32, 100, [900], 128, [71], 4),
], ids=str)
def test_form_for_few_rows_where_the_rule_takes_tiles(E, Hq, Hk, d, Nq, lens, page, q_lens, n):
    """full_tiles False: attention by tiles of 16 rows for any number of them; scores and weights
    of so many are refused, and of few the rule's own bits."""
    p = Problem(Hq, Hk, d, Nq, lens, page, q_lens, seed=526)
    lists = p.lists(n, seed=4)
    p.check_blocks(E, lists, full_tiles=False)
    b, lse = torch.zeros(p.n_pages, Hk, 2, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(p.q.shape[:3], device="cuda")
    args = p.table.cuda(), p.lens.cuda()
    with pytest.raises(E.AttnError, match="few rows"):
        E.block_scores(p.q.cuda(), b, *args, page_size=page, full_tiles=False)
    with pytest.raises(E.AttnError, match="few rows"):
        E.kv_weights(p.q.cuda(), p.k.cuda(), *args, lse, p.w.cuda(), full_tiles=False)
    few = Problem(Hq, Hk, d, 2, lens, page, seed=527)
    assert torch.equal(few.check_scores(E, full_tiles=False), few.check_scores(E))
    few.check_weights(E, full_tiles=False)


@FORMS
def test_blocks_of_rising_maxima(E, full):
    """Scores that grow from page to page by far more than the running maximum's slack."""
    p = Problem(4, 1, 64, 1, [900], 16, seed=530)
    ramp = torch.linspace(0.1, 14.0, 57)
    for j, pg in enumerate(p.table[0].tolist()):
        p.k[pg] *= ramp[j]
    p.check_blocks(E, p.lists(57, seed=3), full_tiles=full)
    # the other way round: the last page, partly unused, is then read whole
    p.k, p.v, p.table = p.k0(), p.v.nan_to_num(0.0), p.table.flip(1)
    p.lens = ints([56 * 16])
    p.check_blocks(E, torch.arange(57, dtype=torch.int32).expand(1, 1, 1, 57).contiguous(), full_tiles=full)


@FORMS
def test_blocks_with_scores_that_are_not_finite(E, full):
    """A key of NaN or a score of +inf gives NaN where it is read, nothing where it is not;
    a row of scores -inf is a row without a key."""
    p = Problem(2, 1, 64, 1, [64], 16, seed=540)
    p.q = p.q.abs() + 1
    ids = p.table[0].tolist()
    p.k[ids[0], :, 2], p.k[ids[1], :, 5], p.k[ids[2], :] = float("nan"), float("inf"), -float("inf")
    for entry, want in ((0, "nan"), (1, "nan"), (2, "none"), (3, "fine")):
        o, lse = p.run_blocks(E, ints([[[[entry, -1]]]]), full_tiles=full)
        if want == "nan":
            assert bool(o.isnan().all()) and bool(lse.isnan().all())
        elif want == "none":
            assert bool((o == 0).all()) and bool((lse == -math.inf).all())
        else:
            assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())


@FORMS
def test_weights_of_rows_without_a_sum(E, full):
    """Rows whose lse is -inf count nothing, NaN reaches only the slots that such a row sees."""
    p = Problem(2, 2, 64, 3, [50, 40], 16, seed=550)
    lse = torch.full((2, 2, 3), 2.5)
    lse[0, 0], lse[1, 1, 1], lse[1, 0, 2] = -math.inf, -math.inf, math.inf
    p.check_weights(E, lse=lse, full_tiles=full)
    lse[0, 1, 0] = float("nan")
    w = p.w.cuda()
    E.kv_weights(p.q.cuda(), p.k.cuda(), p.table.cuda(), p.lens.cuda(), lse.cuda(), w, full_tiles=full)
    got = O.rows(w.cpu(), p.table[0], 50)
    assert bool(got[1, :48].isnan().all()) and not bool(got[1, 48:].isnan().any()) and not bool(got[0].isnan().any())


@FORMS
def test_weights_of_infinite_products_and_lse(E, full):
    """exp(s - lse) with an infinity on either side, or on both: 0, infinity, NaN in every form."""
    p = Problem(4, 1, 32, 1, [40], 16, seed=561)
    p.q = p.q.abs() + 1
    page = int(p.table[0, 0])
    p.k[page, 0, 3], p.k[page, 0, 4] = float("inf"), -float("inf")
    inf = math.inf
    most = torch.finfo(torch.float32).max
    for row, want3, want4 in ((inf, "nan", 0.0), (-inf, 0.0, 0.0), (3.0, inf, 0.0), (1e38, inf, 0.0), (-1e38, inf, 0.0),
                              (most, inf, 0.0), (-most, inf, 0.0)):
        lse = torch.full((1, 4, 1), -inf)
        lse[0, 1] = row
        w = p.w.cuda()
        E.kv_weights(p.q.cuda(), p.k.cuda(), p.table.cuda(), p.lens.cuda(), lse.cuda(), w, decay=0.0, full_tiles=full)
        got = O.rows(w.cpu(), p.table[0], 40)[0]
        for at, want in ((3, want3), (4, want4)):
            assert bool(got[at].isnan()) if want == "nan" else float(got[at]) == want, (row, at, float(got[at]))
        rest = got[[0, 1, 2, 5, 39]]
        assert bool((rest == (inf if -inf < row < 0 else 0.0)).all()) if row != 3.0 else bool(torch.isfinite(rest).all())


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Hq,Hk,Nq", [(3, 1, 700), (16, 2, 130), (1, 1, 1)])
def test_weights_of_many_tiles_of_rows(E, d, Hq, Hk, Nq):
    """Dozens of tiles of 64 rows go through the few stages of shared memory."""
    Problem(Hq, Hk, d, Nq, [Nq + 150, Nq], 16, [Nq, max(1, Nq - 60)], seed=640).check_weights(E, full_tiles=True)


@FORMS
def test_weights_of_keys_that_are_infinite(E, full):
    p = Problem(1, 1, 32, 1, [40], 16, seed=560)
    p.q = p.q.abs() + 1
    p.k[int(p.table[0, 0]), 0, 3] = -float("inf")
    w = p.w.cuda()
    E.kv_weights(p.q.cuda(), p.k.cuda(), p.table.cuda(), p.lens.cuda(), torch.full((1, 1, 1), 3.0).cuda(), w, decay=0.0,
                 full_tiles=full)
    assert float(w[int(p.table[0, 0]), 0, 3]) == 0.0 and bool(torch.isfinite(O.rows(w.cpu(), p.table[0], 40)).all())


@FORMS
@pytest.mark.parametrize("d", [32, 64, 128])
def test_weights_sum_to_the_number_of_rows(E, d, full):
    """With the lse that the attention returned, each row hands out one in all."""
    p = Problem(6, 2, d, 20, [20, 300, 77], 32, [20, 13, 1], seed=570)
    args = p.k.cuda(), p.v.cuda(), p.table.cuda(), p.lens.cuda()
    _, lse = E.attn_paged(p.q.cuda(), *args, q_lens=p.q_lens.cuda())
    w = p.w.cuda()
    E.kv_weights(p.q.cuda(), args[0], args[2], args[3], lse, w, q_lens=p.q_lens.cuda(), decay=0.0, full_tiles=full)
    for b in range(3):
        got = O.rows(w.cpu(), p.table[b], int(p.lens[b])).sum(1)
        assert torch.allclose(got, torch.full((2,), 3.0 * int(p.q_lens[b])).double(), rtol=2.0 ** -14)


def test_weights_to_another_buffer(E):
    p = Problem(4, 2, 64, 2, [50, 70], 16, seed=580)
    lse, out = torch.full((2, 4, 2), 3.0), rnd(581, p.n_pages, 2, 16).float()
    w, to = p.w.cuda(), out.cuda()
    E.kv_weights(p.q.cuda(), p.k.cuda(), p.table.cuda(), p.lens.cuda(), lse.cuda(), w, out=to, decay=0.5)
    assert torch.equal(w.cpu().nan_to_num(0.0), p.w.nan_to_num(0.0))
    ref, err = O.weights(p.q, p.k0(), p.table, p.lens, lse, p.w, None, p.scale, "causal_br", 0.5, out=out)
    check("weights", to, ref, err)


def evicted(E, p, budget, first, last, dst=None):
    k, v, w = p.k.cuda(), p.v.cuda(), p.w.cuda()
    lens, kept = E.kv_evict(k, v, w, p.table.cuda(), p.lens.cuda(), budget, first=first, last=last,
                            dst_table=None if dst is None else dst.cuda())
    rk, rv, rw, rl, rkept = O.evict(p.k, p.v, p.w, p.table, p.lens, budget, first, last, dst)
    assert torch.equal(lens.cpu(), rl) and torch.equal(kept.cpu(), rkept)
    for got, ref in ((k, rk), (v, rv), (w, rw)):
        assert torch.equal(got.cpu().nan_to_num(77.0), ref.nan_to_num(77.0))
    return k, v, w, lens


@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (16, 0, 0), (17, 4, 8), (64, 64, 0), (100, 1, 99), (100, 7, 13),
                                               (300, 0, 30), (1000, 5, 5)])
@pytest.mark.parametrize("Hk,d,page", [(1, 32, 16), (3, 64, 16), (2, 128, 64)])
def test_evict(E, Hk, d, page, budget, first, last):
    lens = [0, 1, 17, 100, 101, 330, 64]
    need = -(-min(budget, 330) // page)
    p = Problem(Hk, Hk, d, 1, lens, page, seed=600, spare=need * len(lens) + 1)
    evicted(E, p, budget, first, last)
    evicted(E, p, budget, first, last, p.spare[:need * len(lens)].reshape(len(lens), need))


def test_evict_ties_and_values_that_are_not_finite(E):
    p = Problem(1, 1, 32, 1, [200, 333], 16, seed=610)
    p.w = torch.where(p.w.isnan(), p.w, (p.w * 1.5).round())
    for at, x in ((3, float("nan")), (50, math.inf), (51, -math.inf), (52, -0.0), (53, 0.0)):
        p.w[int(p.table[0, at // 16]), 0, at % 16] = x
    evicted(E, p, 70, 0, 0)
    evicted(E, p, 160, 1, 3)


@pytest.mark.parametrize("n", [4096, 4097, 16384, 16385, 32768, 32769, 70000])
def test_evict_long(E, n):
    """Lengths around the sizes of the teams that share a row."""
    p = Problem(1, 1, 32, 1, [n, n // 3], 16, seed=620)
    p.w = torch.where(p.w.isnan(), p.w, (p.w * 1000).round())
    evicted(E, p, 1000, 3, 20)


def test_evict_where_the_table_names_no_page(E):
    """Missing sources read as zeros, missing destinations are left out."""
    p = Problem(2, 2, 64, 1, [100, 90], 16, seed=630, spare=9)
    p.table[0, 2], p.table[1, 0] = -1, p.n_pages
    evicted(E, p, 50, 2, 5)
    dst = p.spare[:8].reshape(2, 4).clone()
    dst[0, 1], dst[1, 3] = -3, 1 << 29
    evicted(E, p, 50, 2, 5, dst)


@FORMS
def test_lengths_beyond_the_table_are_cut(E, full):
    p = Problem(2, 1, 32, 1, [48, 20], 16, seed=640)
    p.lens = ints([1 << 30, -5])
    p.check_scores(E, full_tiles=full)
    p.check_blocks(E, p.lists(6), full_tiles=full)
    p.check_weights(E, full_tiles=full)
    evicted(E, p, 20, 1, 1)


@FORMS
def test_pages_that_the_cache_has_not(E, full):
    """Entries that name no page read as zeros: scores and values 0, nothing outside."""
    p = Problem(2, 1, 64, 1, [64], 16, seed=650)
    p.table[0, 1], p.table[0, 3] = p.n_pages, -1
    p.check_scores(E, full_tiles=full)
    p.check_blocks(E, ints([[[[0, 1, 2, 3]]]]), full_tiles=full)
    p.check_weights(E, full_tiles=full)


def sharing(Hq, Hk, d, Nq, own, page, shared, seed, spare=1):
    """Sequences whose first `shared` pages are the first one's; the others' stay unused."""
    p = Problem(Hq, Hk, d, Nq, [shared * page + n for n in own], page, seed=seed, spare=spare)
    p.table[1:, :shared] = p.table[:1, :shared]
    return p


@FORMS
@pytest.mark.parametrize("Hq,Hk,d,Nq,page", [(4, 2, 64, 1, 16), (6, 2, 128, 7, 64), (2, 1, 32, 40, 32)], ids=str)
def test_pages_that_sequences_share(E, Hq, Hk, d, Nq, page, full):
    """A prefix's pages in every row of the table: bounds, scores, choice and attention."""
    p = sharing(Hq, Hk, d, Nq, [Nq + 3, Nq + 100, Nq], page, 5, seed=653)
    s = p.check_scores(E, full_tiles=full)
    lists = E.block_select(s, p.lens.cuda(), 4, page_size=page)
    assert torch.equal(lists.cpu(), O.select(s.cpu(), p.lens, None, 4, page, 1, 2, "causal_br"))
    p.check_blocks(E, lists.cpu(), full_tiles=full)


@FORMS
def test_weights_and_eviction_with_a_shared_prefix(E, full):
    """What their documentation says: a call for each sequence, and pages of its own for each."""
    p = sharing(4, 2, 64, 3, [40, 9, 3], 16, 4, seed=654, spare=13)
    lse = 2 + torch.rand(3, 4, 3, generator=torch.Generator().manual_seed(9))
    w = p.w.cuda() * 0.5
    ref, err = p.w.double() * 0.5, torch.zeros(p.w.shape, dtype=torch.float64)
    for b in range(3):
        one = slice(b, b + 1)
        E.kv_weights(p.q[one].cuda(), p.k.cuda(), p.table[one].cuda(), p.lens[one].cuda(), lse[one].cuda(), w, full_tiles=full)
        ref, e = O.weights(p.q[one], p.k0(), p.table[one], p.lens[one], lse[one], ref, None, p.scale, "causal_br", 1.0)
        err += e
    done(E)
    check("weights", w.cpu().nan_to_num(0.0), ref.nan_to_num(0.0), err)
    p.w = w.cpu()
    evicted(E, p, 50, 3, 10, p.spare[:12].reshape(3, 4))


def test_timeouts_are_reported(E):
    """Something withheld in the forms with tiles of 128 rows: the bounded wait runs out, the
    status says so, and the next call is right."""
    p = Problem(4, 1, 64, 40, [700], 16, seed=655)
    lists, how = p.lists(5), dict(timeout_ns=20_000_000, inject=1, full_tiles=True)
    b = torch.zeros(p.n_pages, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    args = p.table.cuda(), p.lens.cuda()
    for call in (lambda: p.run_blocks(E, lists, **how), lambda: E.block_scores(p.q.cuda(), b, *args, page_size=16, **how),
                 lambda: E.kv_weights(p.q.cuda(), p.k.cuda(), *args, torch.zeros(1, 4, 40).cuda(), p.w.cuda(), **how)):
        call()
        torch.cuda.synchronize()
        code, detail = E.device_status()
        assert code == 5 and detail[0] == 5
        p.check_blocks(E, lists, full_tiles=True)
        p.check_scores(E, full_tiles=True)
        p.check_weights(E, full_tiles=True)


@pytest.mark.parametrize("Nq", [10, 40])
def test_scores_that_give_up(E, Nq):
    """The wait that runs out is the only one (40 rows, one tile), or one between tiles."""
    p = Problem(4, 2, 64, Nq, [700, 90], 16, seed=656)
    b = torch.zeros(p.n_pages, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        E.block_scores(p.q.cuda(), b, p.table.cuda(), p.lens.cuda(), page_size=16, full_tiles=True, timeout_ns=1, inject=1)
        torch.cuda.synchronize()
        code, detail = E.device_status()
        assert code == 5 and detail[0] == 5
        p.check_scores(E, full_tiles=True)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Nq", [10, 40, 200])
def test_weights_that_give_up(E, Nq, d):
    """All products issued (one tile, two), or some: whichever warp's wait runs out, the block
    waits for its products, writes no weight and leaves nothing behind for the next call."""
    p = Problem(4, 2, d, Nq, [700, 290], 16, seed=657)
    for _ in range(2):
        w = torch.zeros(p.n_pages, 2, 16, device="cuda")
        E.kv_weights(p.q.cuda(), p.k.cuda(), p.table.cuda(), p.lens.cuda(), torch.zeros(2, 4, Nq).cuda(), w, decay=0.0,
                     full_tiles=True, timeout_ns=1, inject=1)
        torch.cuda.synchronize()
        code, detail = E.device_status()
        assert code == 5 and detail[0] == 5 and not bool(w.any())
        p.check_weights(E, full_tiles=True)


def test_layouts(E):
    """Heads-last queries and outputs, [page, slot, head, d] caches, K and V in one tensor, a
    wider table."""
    p = Problem(6, 3, 64, 4, [77, 210], 32, seed=660)
    q, table, lens, lists = p.q.cuda(), p.table.cuda(), p.lens.cuda(), p.lists(5).cuda()
    want = p.run_blocks(E, lists)
    qh = q.transpose(1, 2).contiguous().transpose(1, 2)
    kn, vn = (t.cuda().transpose(1, 2).contiguous().transpose(1, 2) for t in (p.k, p.v))
    wide = torch.full((2, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out = torch.empty(2, 4, 6, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    o = E.attn_blocks(qh, kn, vn, wide[:, :table.shape[1]], lens, lists, out=out, return_lse=False)
    assert o.data_ptr() == out.data_ptr() and torch.equal(o, want[0])
    kv = torch.stack([p.k, p.v], dim=1).cuda()
    got = E.attn_blocks(q, kv[:, 0], kv[:, 1], table, lens, lists)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    lse = torch.full((2, 6, 4), 3.0, device="cuda")
    w1, w2 = p.w.cuda(), p.w.cuda()
    assert torch.equal(E.attn_blocks(qh, kn, vn, wide[:, :table.shape[1]], lens, lists, full_tiles=True)[0],
                       p.run_blocks(E, lists, full_tiles=True)[0])
    E.kv_weights(q, p.k.cuda(), table, lens, lse, w1)
    E.kv_weights(qh, kn, wide[:, :table.shape[1]], lens, lse, w2)
    assert torch.equal(w1.nan_to_num(0.0), w2.nan_to_num(0.0))
    b1, b2 = (torch.zeros(p.n_pages, 3, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    E.kv_bounds(p.k.cuda(), b1, table, lens)
    E.kv_bounds(kn, b2, wide, lens)
    assert torch.equal(b1, b2)
    s1 = E.block_scores(q, b1, table, lens, page_size=32)
    s2 = E.block_scores(qh, b1, wide, lens, page_size=32)
    assert torch.equal(s1, s2[..., :table.shape[1]]) and bool((s2[..., table.shape[1]:] == -math.inf).all())
    k1, v1, wa = p.k.cuda(), p.v.cuda(), p.w.cuda()
    wb = p.w.cuda()
    E.kv_evict(k1, v1, wa, table, lens, 40, last=9)
    E.kv_evict(kn, vn, wb, table, lens, 40, last=9)
    assert torch.equal(kn.nan_to_num(0.0), k1.nan_to_num(0.0)) and torch.equal(vn.nan_to_num(0.0), v1.nan_to_num(0.0))


def step(E, p, bnd, w, n=4, stream=None, full=None, **bufs):
    """One decoding step of every operator, into given buffers."""
    kw = dict(stream=stream, full_tiles=full)
    E.kv_bounds(bufs["k"], bnd, bufs["table"], bufs["lens"], n_new=p.Nq, stream=stream)
    s = E.block_scores(bufs["q"], bnd, bufs["table"], bufs["lens"], page_size=p.page, **kw)
    lists = E.block_select(s, bufs["lens"], n, page_size=p.page, stream=stream)
    o, lse = E.attn_blocks(bufs["q"], bufs["k"], bufs["v"], bufs["table"], bufs["lens"], lists, **kw)
    E.kv_weights(bufs["q"], bufs["k"], bufs["table"], bufs["lens"], lse, w, **kw)
    return s, lists, o, lse


def buffers(p):
    bnd = torch.zeros(p.n_pages, p.Hk, 2, p.d, dtype=torch.bfloat16)
    return (O.bounds(p.k, bnd, p.table, p.lens, None).cuda(), p.w.cuda(),
            dict(q=p.q.cuda(), k=p.k.cuda(), v=p.v.cuda(), table=p.table.cuda(), lens=p.lens.cuda()))


@FORMS
def test_same_bits_twice_and_two_streams(E, full):
    """No atomics that change results: equal bits, also for two calls at once."""
    ps = [Problem(8, 2, 128, 1, [100, 700, 33], 16, seed=700), Problem(4, 4, 64, 3, [10, 900], 64, seed=701)]
    want = []
    for p in ps:
        bnd, w, bufs = buffers(p)
        want.append((*step(E, p, bnd, w, full=full, **bufs), w))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        state = [buffers(p) for p in ps]
        torch.cuda.synchronize()
        got = [(*step(E, p, bnd, w, stream=st, full=full, **bufs), w) for p, st, (bnd, w, bufs) in zip(ps, streams, state)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x.nan_to_num(0.0) if x.is_floating_point() else x,
                                   y.nan_to_num(0.0) if y.is_floating_point() else y) for x, y in zip(a, b))


@FORMS
def test_graph_follows_the_lengths(E, full):
    p = Problem(4, 2, 64, 1, [300, 300, 300], 32, seed=800)
    bnd, w, bufs = buffers(p)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s, lists, o, lse = step(E, p, bnd, w, full=full, **bufs)
        new, kept = E.kv_evict(bufs["k"].clone(), bufs["v"].clone(), w.clone(), bufs["table"], bufs["lens"], 100, last=10)
    for now in ([300, 300, 300], [1, 128, 257], [0, 0, 5]):
        bufs["lens"].copy_(ints(now))
        w.copy_(p.w)
        bnd.copy_(O.bounds(p.k, bnd.cpu(), p.table, now, None))
        g.replay()
        torch.cuda.synchronize()
        rs, bs = O.scores(p.q, bnd.cpu(), p.table, now, None, 32, p.scale, "causal_br")
        check("scores", s, rs, bs)
        assert torch.equal(lists.cpu(), O.select(s.cpu(), now, None, 4, 32, 1, 2, "causal_br"))
        ro, bo, rl, bl = O.blocks(p.q, p.k0(), p.v.nan_to_num(0.0), p.table, now, lists.cpu(), None, p.scale, "causal_br")
        check("o", o, ro, bo)
        check("lse", lse, rl, bl)
        assert new.tolist() == [min(n, 100) for n in now]


def test_first_calls_captured():
    """In a new process the first call of each operator may be a captured one."""
    code = """
import torch, exact_attention_69_gb300 as E
t = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")
kc, vc, q, bnd = t(4, 2, 16, 64), t(4, 2, 16, 64), t(2, 4, 1, 64), t(4, 2, 2, 64)
w = torch.ones(4, 2, 16, device="cuda")
table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
lens = torch.tensor([20, 31], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    E.kv_bounds(kc, bnd, table, lens, n_new=1)
    s = E.block_scores(q, bnd, table, lens, page_size=16)
    b = E.block_select(s, lens, 2, page_size=16, first=1, last=1)
    o, lse = E.attn_blocks(q, kc, vc, table, lens, b)
    E.kv_weights(q, kc, table, lens, lse, w)
    new, kept = E.kv_evict(kc, vc, w, table, lens, 18, last=2)
g.replay()
torch.cuda.synchronize()
assert bool((o == 1).all()) and new.tolist() == [18, 18] and b.flatten().tolist() == [0, 1] * 4
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_offsets_beyond_32_bits(E):
    """Caches of more than 2^31 elements: their last pages are read and written."""
    Hk, page, d, n_pages = 8, 64, 128, 33000
    kc, vc = (torch.empty(n_pages, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    ids = [n_pages - 1, 3, n_pages - 2, n_pages - 3]
    p = Problem(Hk, Hk, d, 1, [100, 77], page, seed=900, spare=0)
    big = ints([[ids[int(x)] if 0 <= x < 4 else -1 for x in row] for row in p.table])
    w = torch.empty(n_pages, Hk, page, device="cuda")
    bnd = torch.zeros(n_pages, Hk, 2, d, dtype=torch.bfloat16, device="cuda")
    for i, pg in enumerate(ids):
        kc[pg], vc[pg], w[pg] = p.k[i].cuda(), p.v[i].cuda(), p.w[i].cuda()
    args, lists = (big.cuda(), p.lens.cuda()), p.lists(3)
    o, lse = E.attn_blocks(p.q.cuda(), kc, vc, *args, lists.cuda())
    ro, bo, rl, bl = O.blocks(p.q, p.k0(), p.v.nan_to_num(0.0), p.table, p.lens, lists, None, p.scale, "causal_br")
    check("o", o, ro, bo)
    E.kv_bounds(kc, bnd, *args)
    want = O.bounds(p.k, torch.zeros(4, Hk, 2, d, dtype=torch.bfloat16), p.table, p.lens, None)
    assert torch.equal(bnd[ids].cpu(), want)
    s = E.block_scores(p.q.cuda(), bnd, *args, page_size=page)
    check("scores", s, *O.scores(p.q, want, p.table, p.lens, None, page, p.scale, "causal_br"))
    z = torch.full((2, Hk, 1), 3.0)
    E.kv_weights(p.q.cuda(), kc, *args, z.cuda(), w)
    ref, err = O.weights(p.q, p.k0(), p.table, p.lens, z, p.w, None, p.scale, "causal_br", 1.0)
    check("weights", w[ids].nan_to_num(0.0), ref.nan_to_num(0.0), err)
    rk, rv, rw, rl, rkept = O.evict(p.k, p.v, w[ids].cpu(), p.table, p.lens, 60, 1, 2)
    new, kept = E.kv_evict(kc, vc, w, *args, 60, first=1, last=2)
    assert torch.equal(kept.cpu(), rkept) and torch.equal(kc[ids].cpu().nan_to_num(0.0), rk.nan_to_num(0.0))
    assert torch.equal(vc[ids].cpu().nan_to_num(0.0), rv.nan_to_num(0.0))


@FORMS
@pytest.mark.parametrize("seed", range(16))
def test_random_problems(E, seed, full):
    r = random.Random(seed)
    Hk, G, d = r.choice([1, 2, 3]), r.choice([1, 2, 3, 4, 5, 8, 16, 20]), r.choice([32, 64, 128])
    Nq = r.choice([1, 1, 2, r.randint(3, 20), r.randint(60, 140)])
    B = r.randint(1, 6 if Nq < 21 else 2)
    page = r.choice([16, 32, 64, 128, 512])
    q_lens = [r.randint(0, Nq) for _ in range(B)] if r.random() < 0.4 else None
    lens = [max(r.choice([0, 1, r.randint(2, 900)]), q_lens[b] if q_lens else Nq) if r.random() < 0.8 else r.randint(0, 40)
            for b in range(B)]
    p = Problem(Hk * G, Hk, d, Nq, lens, page, q_lens, seed=2000 + 10 * seed, width=r.choice([None, 40]))
    mask = r.choice(["none", "causal_br"])
    s = p.check_scores(E, mask, full_tiles=full)
    n = r.randint(3, 20)
    lists = E.block_select(s, p.lens.cuda(), n, page_size=page, q_lens=None if q_lens is None else p.q_lens.cuda(), mask=mask)
    assert torch.equal(lists.cpu(), O.select(s.cpu(), p.lens, p.q_lens, n, page, 1, 2, mask))
    p.check_blocks(E, lists.cpu(), mask, full_tiles=full)
    p.check_blocks(E, p.lists(n, seed=seed), mask, full_tiles=full)
    p.check_weights(E, mask, r.choice([0.0, 1.0, 0.75]), full_tiles=full)
    budget = r.randint(1, 400)
    evicted(E, p, budget, r.randint(0, budget // 3), r.randint(0, budget // 3))


def test_refusals(E):
    """What the host can see is refused before anything runs."""
    p = Problem(4, 2, 64, 2, [30, 9], 16, seed=1400)
    bnd, w, b = buffers(p)
    lse, lists = torch.zeros(2, 4, 2, device="cuda"), p.lists(3).cuda()
    s = torch.zeros(2, 2, 2, 2, device="cuda")
    base = dict(
        kv_bounds=dict(k_cache=b["k"], bounds=bnd, block_table=b["table"], kv_lens=b["lens"]),
        block_scores=dict(q=b["q"], bounds=bnd, block_table=b["table"], kv_lens=b["lens"], page_size=16),
        block_select=dict(scores=s, kv_lens=b["lens"], n=2, page_size=16, first=1, last=1),
        attn_blocks=dict(q=b["q"], k_cache=b["k"], v_cache=b["v"], block_table=b["table"], kv_lens=b["lens"], blocks=lists),
        kv_weights=dict(q=b["q"], k_cache=b["k"], block_table=b["table"], kv_lens=b["lens"], lse=lse, weights=w),
        kv_evict=dict(k_cache=b["k"], v_cache=b["v"], weights=w, block_table=b["table"], kv_lens=b["lens"], budget=8))
    bad = dict(
        kv_bounds=[dict(bounds=bnd.float()), dict(bounds=bnd[:1]), dict(k_cache=b["k"].float()), dict(kv_lens=b["lens"].long()),
                   dict(n_new=-2), dict(bounds=bnd.cpu()), dict(block_table=b["table"][:1])],
        block_scores=[dict(q=b["q"].float()), dict(page_size=24), dict(scale=0.0), dict(scale=float("nan")), dict(mask="causal"),
                      dict(out=s[:1]), dict(q=b["q"][:, :3].contiguous()), dict(q_lens=b["lens"].float()), dict(bounds=bnd[:, :, :1])],
        block_select=[dict(n=0), dict(first=2), dict(last=-1), dict(scores=s.double()), dict(scores=s.transpose(2, 3)),
                      dict(page_size=8), dict(n=1 << 40), dict(kv_lens=b["lens"][:1]), dict(mask="wrap")],
        attn_blocks=[dict(blocks=lists.long()), dict(blocks=lists[..., :0]), dict(blocks=lists[:, :1]), dict(scale=-1.0),
                     dict(v_cache=b["v"][:, :1]), dict(lse=lse.double()), dict(out=b["q"][:1]), dict(q=b["q"].cpu()),
                     dict(q=b["q"][..., :32]), dict(inject=2), dict(timeout_ns=-1), dict(timeout_ns=1 << 64)],
        kv_weights=[dict(decay=-0.5), dict(decay=float("inf")), dict(weights=w.double()), dict(lse=lse[:1]), dict(out=w[:1]),
                    dict(weights=w.transpose(0, 1)), dict(lse=lse.cpu()), dict(scale=1e-44)],
        kv_evict=[dict(budget=0), dict(first=5, last=4), dict(weights=w[:1]), dict(dst_table=b["table"].long()),
                  dict(dst_table=b["table"][:1]), dict(v_cache=b["v"].float()), dict(k_cache=b["k"][:1].expand(p.n_pages, -1, -1, -1)),
                  dict(budget=20, dst_table=b["table"][:, :1].contiguous())])
    for name, cases in bad.items():
        getattr(E, name)(**base[name])
        for change in cases:
            with pytest.raises((TypeError, ValueError, E.AttnError)):
                getattr(E, name)(**{**base[name], **change})


def test_written_tensors_are_told_to_autograd(E):
    """A graph that saved a tensor which a call then writes refuses its backward pass."""
    p = Problem(2, 1, 32, 1, [40], 16, seed=1500)
    bnd, w, b = buffers(p)
    w = w.nan_to_num(1.0).requires_grad_(True)
    x = torch.ones_like(w, requires_grad=True)
    loss = (w.detach() * x).sum()
    saved = w.detach()
    y = (saved * x).sum()
    E.kv_weights(b["q"], b["k"], b["table"], b["lens"], torch.zeros(1, 2, 1, device="cuda"), saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    del loss


def test_serving_steps(E):
    """A server's life with a long cache: append, bounds, selection and attention over it,
    weights, eviction when the budget is passed, and on, against the same steps in 64 bits."""
    B, Hq, Hk, d, page, budget, n = 3, 6, 2, 64, 16, 96, 5
    p = Problem(Hq, Hk, d, 1, [160, 160, 160], page, seed=1100)
    kc, vc, table = p.k.cuda(), p.v.cuda(), p.table.cuda()
    w = p.w.cuda()
    bnd = torch.zeros(p.n_pages, Hk, 2, d, dtype=torch.bfloat16, device="cuda")
    held, pos = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    freqs = E.rope_freqs(d)
    for turn, (N, counts) in enumerate([(70, [70, 41, 66]), (1, None), (60, [58, 60, 2]), (1, None), (1, None)]):
        x = rnd(1200 + turn, B, N, Hq + 2 * Hk, d).cuda()
        q, k, v = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2), x[:, :, Hq + Hk:].transpose(1, 2)
        new = ints(counts if counts else [N] * B)
        cnt = new.cuda() if counts else None
        where = (pos[:, None] + torch.arange(N, dtype=torch.int32)).cuda()  # true positions, also after an eviction
        qr = E.kv_append(k, v, kc, vc, table, held.cuda(), counts=cnt, positions=where, inv_freq=freqs, q=q)
        held, pos = held + new, pos + new
        lens = held.cuda()
        E.kv_bounds(kc, bnd, table, lens, n_new=N)
        s = E.block_scores(qr, bnd, table, lens, page_size=page, q_lens=cnt)
        lists = E.block_select(s, lens, n, page_size=page, q_lens=cnt)
        o, lse = E.attn_blocks(qr, kc, vc, table, lens, lists, q_lens=cnt)
        before = w.clone()
        E.kv_weights(qr, kc, table, lens, lse, w, q_lens=cnt)
        # each step is held to what the cache had
        k64, v64, ql = kc.cpu().nan_to_num(0.0), vc.cpu().nan_to_num(0.0), None if cnt is None else new
        assert torch.equal(bnd.cpu(), O.bounds(kc.cpu(), bnd.cpu(), p.table, held, None))
        check("scores", s, *O.scores(qr.cpu(), bnd.cpu(), p.table, held, ql, page, p.scale, "causal_br"))
        assert torch.equal(lists.cpu(), O.select(s.cpu(), held, ql, n, page, 1, 2, "causal_br"))
        ro, bo, rl, bl = O.blocks(qr.cpu(), k64, v64, p.table, held, lists.cpu(), ql, p.scale, "causal_br")
        check("o", o, ro, bo)
        check("lse", lse, rl, bl)
        ref, err = O.weights(qr.cpu(), k64, p.table, held, lse.cpu(), before.cpu(), ql, p.scale, "causal_br", 1.0)
        check("weights", w.cpu().nan_to_num(0.0), ref.nan_to_num(0.0), err)
        if int(held.max()) > budget:
            old = kc.cpu(), vc.cpu(), w.cpu()
            new_lens, kept = E.kv_evict(kc, vc, w, table, lens, budget, first=4, last=16)
            rk, rv, rw, rl, rkept = O.evict(*old, p.table, held, budget, 4, 16)
            assert torch.equal(kept.cpu(), rkept) and torch.equal(kc.cpu().nan_to_num(0.0), rk.nan_to_num(0.0))
            assert torch.equal(w.cpu().nan_to_num(0.0), rw.nan_to_num(0.0))
            held = new_lens.cpu()
            E.kv_bounds(kc, bnd, table, new_lens)
