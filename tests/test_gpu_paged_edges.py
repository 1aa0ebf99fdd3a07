"""GPU: paged attention where its arithmetic is at an edge: maxima that jump inside a
tile. Against the definition in 64 bits (bounds in cache_oracle)."""
import math

import pytest
import torch

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
