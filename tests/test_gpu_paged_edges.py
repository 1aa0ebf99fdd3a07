"""GPU: paged attention where its arithmetic is at an edge: maxima that jump inside a
tile, weights rounded, NaN and infinities in keys and queries that are seen, and forms
that its callers meet less often. Against the definition in 64 bits (bounds in
cache_oracle)."""
import math

import pytest
import torch

from tests import cache_oracle as O
from tests.test_gpu_paged import E, Problem  # noqa: F401  (E: fixture)

pytestmark = pytest.mark.gpu


def stairs(p, Hq, Hk, d, step, rising):
    """Keys along one direction u, scores along u rise by `step` (log2 units) every 64
    keys, prefix and own keys in turn; queries near +u see them rise, near -u fall.
    rising(row) says which, row = query * group + head of the group."""
    g = torch.Generator().manual_seed(77)
    u = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    unit = step / (math.sqrt(d) * math.log2(math.e))  # q.k / sqrt(d) in log2 units, q = u, k = unit * u
    page = p.k.shape[2]
    noise = 0.02 * torch.randn(p.k.shape, generator=g)
    new = torch.full(p.k.shape, float("nan"))
    for b in range(p.q.shape[0]):
        for j in range(p.P + int(p.lens[b])):
            pg = int(p.prefix[j // page] if j < p.P else p.table[b, (j - p.P) // page])
            at = (j if j < p.P else j - p.P) % page
            new[pg, :, at] = (j // 64) * unit * u + noise[pg, :, at]
    p.k = new.to(torch.bfloat16)
    B, _, Nq, _ = p.q.shape
    G = Hq // Hk
    sign = torch.tensor([[1.0 if rising(n * G + h % G) else -1.0 for n in range(Nq)] for h in range(Hq)])
    p.q = (sign[None, :, :, None] * u + 0.05 * torch.randn(p.q.shape, generator=g)).to(torch.bfloat16)


@pytest.mark.parametrize("rows", ["all", "one of a warp", "every second"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Hq,Hk,Nq,P,lens", [(4, 1, 1, 0, [1000]), (2, 2, 3, 300, [700, 650]), (2, 1, 90, 128, [900])],
                         ids=["one tile", "one tile, prefix", "two tiles"])
def test_maxima_jump_in_both_halves_of_a_tile(E, Hq, Hk, Nq, P, lens, d, rows):  # noqa: F811
    """Every 64 keys the maximum rises by 12 log2 units, so both halves of every tile, later
    ones too, bring O, the sum and P to a new reference: in tasks of one query tile (tiles
    in turn) and of two, whole in one CTA and cut."""
    p = Problem(Hq, Hk, d, Nq, P, lens, 32, seed=3000 + d)
    stairs(p, Hq, Hk, d, 12.0, {"all": lambda r: True, "one of a warp": lambda r: r % 32 == 2,
                                "every second": lambda r: r % 2 == 0}[rows])
    for ctas in (1, 3):
        p.check(E, num_ctas=ctas)


def check_nan(name, got, ref, bound):
    """As O.check, and NaN where the definition has NaN."""
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in the wrong places"
    rest = ~torch.isnan(ref)
    O.check(name, got[rest], ref[rest], bound[rest])


# whole in one CTA, cut over many, prefix apart from the own keys, pairs of query tiles
NAN_CASES = [(4, 2, 64, 1, 0, [700, 0, 40], 16, 1), (4, 2, 128, 1, 0, [900, 33], 32, 0),
             (8, 2, 64, 1, 600, [(7 * i) % 90 + 1 for i in range(60)], 16, 0),
             (4, 2, 32, 2, 1500, [1, 300, 2], 16, 2), (2, 1, 64, 100, 260, [100, 500], 64, 3)]


@pytest.mark.parametrize("case", NAN_CASES, ids=str)
@pytest.mark.parametrize("where", ["query", "half of a query", "first prefix or own key", "last own key"])
def test_nan_scores_give_nan(E, case, where):  # noqa: F811
    """A score that is NaN and seen makes its row NaN, O and LSE, whatever the cuts are: all
    of a row's scores, or one key's (alone in its part, or far below the other scores)."""
    Hq, Hk, d, Nq, P, lens, page, ctas = case
    p = Problem(Hq, Hk, d, Nq, P, lens, page, seed=3100)
    nan = float("nan")
    if where == "query":
        p.q[0, 1, Nq - 1] = nan
    elif where == "half of a query":
        p.q[-1, :, 0, d // 2:] = nan
    elif where == "first prefix or own key":
        if P:
            p.k[int(p.prefix[0]), 0, 0, 3] = nan
        else:
            p.k[int(p.table[0, 0]), 0, 0, 3] = nan
    else:
        at = lens[-1] - 1
        p.k[int(p.table[-1, at // page]), -1, at % page, 0] = nan
    q, k, v, table, ln, q_lens, prefix = p.cuda()
    o, lse = E.attn_paged(q, k, v, table, ln, q_lens=q_lens, prefix_table=prefix, prefix_len=P, num_ctas=ctas)
    assert E.device_status()[0] == 0
    # (slots that no sequence holds are NaN too: the definition never looks at them)
    ro, bo, rl, bl = O.paged(p.q, p.k, p.v, p.table, p.lens, p.q_lens, p.prefix, P, 1 / math.sqrt(d), "causal_br")
    assert bool(torch.isnan(rl).any())
    check_nan("o", o, ro, bo)
    check_nan("lse", lse, rl, bl)


@pytest.mark.parametrize("ctas", [1, 0])
def test_nan_key_in_a_part_without_weight(E, ctas):  # noqa: F811
    """A NaN key among keys whose weights underflow (scores 300 log2 units lower)."""
    p = Problem(4, 1, 64, 1, 0, [2000], 32, seed=3200)
    stairs(p, 4, 1, 64, 12.0, lambda r: True)
    p.k[int(p.table[0, 0]), 0, 5] = float("nan")
    q, k, v, table, ln, _, _ = p.cuda()
    o, lse = E.attn_paged(q, k, v, table, ln, num_ctas=ctas)
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


def test_infinite_scores(E):  # noqa: F811
    """+inf: NaN for O and LSE. -inf: a key without weight; a row with no other has seen
    nothing."""
    p = Problem(2, 1, 64, 1, 0, [300, 300, 20], 16, seed=3300)
    p.q = p.q.abs() + 0.1
    inf = float("inf")
    p.k[int(p.table[0, 2]), 0, 3] = inf
    p.k[int(p.table[1, 0]), 0, :9] = -inf
    for j in range(20):
        p.k[int(p.table[2, j // 16]), 0, j % 16] = -inf
    # sequence 1 without those keys, in pages of its own
    k1, v1 = (torch.zeros(1, 1, 304, 64, dtype=torch.bfloat16) for _ in range(2))
    for j in range(9, 300):
        at = int(p.table[1, j // 16]), 0, j % 16
        k1[0, 0, j - 9], v1[0, 0, j - 9] = p.k[at], p.v[at]
    ro, bo, rl, bl = O.paged(p.q[1:2], k1, v1, torch.zeros(1, 1, dtype=torch.int32), [291], None, None, 0, 1 / 8, "causal_br")
    for ctas in (1, 0):
        q, k, v, table, ln, _, _ = p.cuda()
        o, lse = E.attn_paged(q, k, v, table, ln, num_ctas=ctas)
        assert bool(torch.isnan(o[0]).all()) and bool(torch.isnan(lse[0]).all())
        assert float(o[2].abs().max()) == 0.0 and bool((lse[2] == -inf).all())
        O.check("o", o[1:2], ro, bo)
        O.check("lse", lse[1:2], rl, bl)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("before", [0, 128, 200])
def test_weights_are_rounded_once(E, d, before):  # noqa: F811
    """Weights that lie just below half a bf16 step, 63 alike, then keys 2^9 times as heavy
    whose ratio lies there too and whose values are 0: rounding the 63 once for their own
    maximum and again for the new one would move O by two half steps. Scores are in log2
    units: scale = ln 2. `before`: lighter keys ahead of them."""
    p = Problem(4, 1, d, 1, 0, [before + 128], 16, seed=3400)
    p.q = torch.zeros_like(p.q)
    p.q[..., :2] = 1.0
    low = torch.tensor(1.4 / 256).to(torch.bfloat16)
    g = torch.arange(d) % 32
    first = before // 64 * 64  # where a half of a tile starts
    for j in range(before + 128):
        at = int(p.table[0, j // 16]), 0, j % 16
        p.k[at] = 0
        p.v[at] = 1 + g / 128.0
        if j < first:
            p.k[at][0] = -30.0
        elif j < first + 64:
            p.k[at][0], p.k[at][1] = (0.0, 0.0) if j == first else (-1.0, low)
        else:
            p.k[at][0], p.k[at][1] = 9.0, -low
            p.v[at] = 0
    q, k, v, table, ln, _, _ = p.cuda()
    k0, v0 = (c.nan_to_num(0.0) for c in (p.k, p.v))
    ro, bo, rl, bl = O.paged(p.q, k0, v0, p.table, p.lens, None, None, 0, math.log(2), "causal_br")
    for ctas in (1, 0):
        o, lse = E.attn_paged(q, k, v, table, ln, scale=math.log(2), num_ctas=ctas)
        O.check("o", o, ro, bo)
        O.check("lse", lse, rl, bl)


@pytest.mark.parametrize("what", ["heads", "queries", "sequences", "scale"])
@pytest.mark.parametrize("case", [(8, 2, 64, 1, 600, [(7 * i) % 90 + 1 for i in range(60)], 16),
                                  (4, 2, 128, 3, 0, [70, 300], 32), (2, 1, 32, 140, 50, [200], 64)], ids=str)
def test_expanded_queries_and_a_scale(E, case, what):  # noqa: F811
    """Queries with a stride of zero over heads, tokens or sequences (gathered row by row), and
    a scale other than 1 / sqrt(d)."""
    Hq, Hk, d, Nq, P, lens, page = case
    p = Problem(Hq, Hk, d, Nq, P, lens, page, seed=3500)
    q, k, v, table, ln, _, prefix = p.cuda()
    scale = 0.31 if what == "scale" else 1 / math.sqrt(d)
    if what != "scale":
        dim = {"sequences": 0, "heads": 1, "queries": 2}[what]
        q = q.narrow(dim, 0, 1).expand(p.q.shape)
    k0, v0 = (c.nan_to_num(0.0) for c in (p.k, p.v))
    ro, bo, rl, bl = O.paged(q.cpu(), k0, v0, p.table, p.lens, None, p.prefix, P, scale, "causal_br")
    for ctas in (0, 2):
        o, lse = E.attn_paged(q, k, v, table, ln, prefix_table=prefix, prefix_len=P, scale=scale, num_ctas=ctas)
        O.check("o", o, ro, bo)
        O.check("lse", lse, rl, bl)


@pytest.mark.parametrize("mask", ["causal_br", "none"])
@pytest.mark.parametrize("ctas", [0, 1, 7])
def test_many_tasks_of_a_sequence(E, ctas, mask):  # noqa: F811
    """Chunks of many tasks (up to 12 of 256 rows a key head), the last ones of some sequences
    without a row, early ones of a causal chunk with few keys."""
    Problem(4, 2, 64, 1500, 130, [1600, 0, 700, 1500], 64, [1500, 0, 257, 1], seed=3600).check(E, mask, num_ctas=ctas)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("at", [0, 5, 135, 300])
def test_a_key_with_all_of_the_weight(E, d, at):  # noqa: F811
    """A key 57 log2 units above the others, in the first half of a tile: its weight is 1
    without a rounding, and O is its value, bit for bit."""
    p = Problem(4, 1, d, 1, 0, [500], 16, seed=3700)
    g = torch.Generator().manual_seed(3701)
    p.q = (1 + torch.rand(p.q.shape, generator=g)).to(torch.bfloat16)
    scale = 40.3 / (float(p.q[0, :, 0].float().sum(-1).min()) * math.log2(math.e))
    for j in range(500):
        p.k[int(p.table[0, j // 16]), 0, j % 16] = 1.0 if j == at else -0.415
    q, k, v, table, ln, _, _ = p.cuda()
    want = p.v[int(p.table[0, at // 16]), 0, at % 16]
    for ctas in (1, 0):
        o, _ = E.attn_paged(q, k, v, table, ln, scale=scale, num_ctas=ctas)
        assert torch.equal(o[0, :, 0].cpu(), want.expand(4, d))
