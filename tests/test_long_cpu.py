"""CPU: refusals of the long-cache entry points (host checks, before any CUDA call), and
the definitions that the kernels are held to against hand-made examples."""
import ctypes
import math

import pytest
import torch

from exact_attention_69_gb300 import _lib
from tests import long_oracle as O

INV, UNS, MIS = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_UNSUPPORTED, _lib.ATTN_ERR_MISALIGNED
A = 1 << 20  # a pointer that no call may touch


@pytest.fixture(scope="module")
def lib():
    from exact_attention_69_gb300 import build
    build.build()
    return _lib.load()


def block(name):
    p = _lib.AttnLongParams()
    given = dict(
        attn_kv_bounds=("k_cache", "bounds"), attn_block_scores=("q", "bounds", "scores"),
        attn_block_select=("scores", "blocks"), attn_blocks=("q", "k_cache", "v_cache", "o", "lse", "blocks"),
        attn_kv_weights=("q", "k_cache", "lse", "weights", "weights_out"),
        attn_kv_evict=("k_cache", "v_cache", "weights", "kept", "new_lens"))[name]
    for n in given + ("block_table",):
        setattr(p, n, A)
    p.kv_lens = 2 * A
    p.B, p.Hq, p.Hk, p.Nq, p.d, p.scale, p.mask_kind = 2, 8, 2, 3, 64, 0.125, _lib.ATTN_MASK_CAUSAL_BR
    p.n_pages, p.page_size, p.table_width, p.table_stride, p.n, p.decay = 9, 16, 4, 4, 8, 1.0
    return p


COMMON = [(dict(B=0), INV), (dict(Hk=0), INV), (dict(B=70000), INV), (dict(page_size=8), INV), (dict(page_size=48), INV),
          (dict(full_tiles=3), INV), (dict(inject=2), INV), (dict(kv_lens=None), INV), (dict(kv_lens=A + 2), MIS), (dict(table_width=0), INV),
          (dict(table_width=1 << 27, table_stride=1 << 27), INV)]
TABLE = [(dict(block_table=None), INV), (dict(block_table=A + 1), MIS), (dict(table_stride=3), INV), (dict(n_pages=0), INV)]
HEADS = [(dict(d=48), UNS), (dict(d=256), UNS)]
QUERIES = [(dict(Nq=0), INV), (dict(mask_kind=_lib.ATTN_MASK_CAUSAL), INV), (dict(q_lens=A + 2), MIS), (dict(B=1 << 15, Nq=1 << 20), INV)]
Q = [(dict(q=None), INV), (dict(q=A + 8), MIS), (dict(Hq=7), INV), (dict(Hq=0), INV), (dict(q_stride=(4096, 512, 60)), MIS),
     (dict(scale=0.0), INV), (dict(scale=math.inf), INV), (dict(q_stride=(4096, -512, 64)), INV)]
KEYS = [(dict(k_cache=None), INV), (dict(k_cache=A + 2), MIS), (dict(k_cache_stride=(2048, 60, 64)), MIS)]
VALUES = [(dict(v_cache=None), INV), (dict(v_cache=A + 4), MIS)]
TAKEN = [(dict(n=0), INV), (dict(first=-1), INV), (dict(last=-1), INV), (dict(first=5, last=4), INV)]
BAD = dict(
    attn_kv_bounds=COMMON + TABLE + HEADS + KEYS + [(dict(bounds=None), INV), (dict(bounds=A + 8), MIS), (dict(n_new=-2), INV)],
    attn_block_scores=COMMON + TABLE + HEADS + QUERIES + Q + [(dict(bounds=None), INV), (dict(bounds=A + 2), MIS), (dict(scores=None), INV),
                                                              (dict(scores=A + 2), MIS)],
    attn_block_select=COMMON + QUERIES + TAKEN + [(dict(scores=None), INV), (dict(blocks=None), INV), (dict(blocks=A + 2), MIS)],
    attn_blocks=COMMON + TABLE + HEADS + QUERIES + Q + KEYS + VALUES + [
        (dict(blocks=None), INV), (dict(o=None), INV), (dict(o=A + 8), MIS), (dict(o_stride=(64, 64, 0)), INV), (dict(n=0), INV),
        (dict(n=1 << 29), INV), (dict(lse=A + 2), MIS)],
    attn_kv_weights=COMMON + TABLE + HEADS + QUERIES + Q + KEYS + [(dict(lse=None), INV), (dict(weights=None), INV),
                                                                   (dict(weights_out=None), INV), (dict(decay=-1.0), INV), (dict(decay=math.nan), INV),
                                                                   (dict(weights=A + 2), MIS), (dict(scale=1e-44), INV), (dict(scale=2.0 ** -65), INV), (dict(scale=2.0 ** 65), INV)],
    attn_kv_evict=COMMON + TABLE + HEADS + KEYS + VALUES + TAKEN + [
        (dict(weights=None), INV), (dict(weights=A + 8), MIS), (dict(kept=None), INV), (dict(new_lens=None), INV), (dict(new_lens=2 * A), INV),
        (dict(k_cache_stride=(1024, 1024, 64)), INV), (dict(v_cache_stride=(64, 1024, 64)), INV), (dict(dst_table=A), INV),
        (dict(dst_table=A, dst_width=2, dst_stride=1), INV), (dict(dst_table=A + 2, dst_width=2, dst_stride=2), MIS),
        (dict(dst_table=A, dst_width=1, dst_stride=1, n=20), INV)],
)


@pytest.mark.parametrize("name,changes,code", [(n, c, e) for n, cases in BAD.items() for c, e in cases], ids=str)
def test_refuses(lib, name, changes, code):
    p = block(name)
    for k, v in changes.items():
        if isinstance(v, tuple):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    assert getattr(lib, name)(ctypes.byref(p)) == code, lib.attn_last_error()
    assert lib.attn_last_error()


@pytest.mark.parametrize("name,G,most", [("attn_block_scores", 1, 32), ("attn_block_scores", 3, 8), ("attn_block_scores", 9, 2),
                                         ("attn_kv_weights", 1, 32), ("attn_kv_weights", 3, 10), ("attn_kv_weights", 9, 3)])
def test_form_for_few_rows(lib, name, G, most):
    """Asked for by name it is refused where it does not hold the rows; else the next check refuses."""
    p = block(name)
    p.Hq, p.full_tiles, p.bounds, p.decay = p.Hk * G, 2, A + 8, -1.0
    p.q_stride[:] = (0, 0, 0)
    for Nq, refused in ((most, False), (most + 1, True), (1 << 20, True)):
        p.Nq = Nq
        code, why = getattr(lib, name)(ctypes.byref(p)), lib.attn_last_error()
        assert code != 0 and (b"few rows" in why if refused else b"aligned" in why or b"decay" in why), (Nq, code, why)


def test_null_blocks(lib):
    for name in _lib.LONG_CALLS:
        assert getattr(lib, name)(None) == INV


def test_python_refuses(lib):
    import exact_attention_69_gb300 as E
    q, w = torch.zeros(1, 2, 16, 32, dtype=torch.bfloat16), torch.zeros(1, 2, 16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        E.kv_bounds(q, q, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        E.block_scores(q, q, table, lens, page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        E.block_select(torch.zeros(1, 1, 1, 1), lens, 4, page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        E.attn_blocks(q, q, q, table, lens, table)
    with pytest.raises(ValueError, match="CUDA"):
        E.kv_weights(q, q, table, lens, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        E.kv_evict(q, q, w, table, lens, 4)
    for bad in (dict(n=0), dict(n=2), dict(n=1 << 32), dict(first=-1), dict(page_size=1 << 40)):
        with pytest.raises(ValueError):
            E.block_select(torch.zeros(1, 1, 1, 1), lens, **{**dict(n=4, page_size=16), **bad})
    for bad in (dict(budget=0), dict(budget=1 << 31), dict(budget=4, last=5)):
        with pytest.raises(ValueError):
            E.kv_evict(q, q, w, table, lens, **bad)
    for bad in (-1.0, math.nan, math.inf):
        with pytest.raises(ValueError, match="decay"):
            E.kv_weights(q, q, table, lens, w, w, decay=bad)
    with pytest.raises(ValueError, match="n_new"):
        E.kv_bounds(q, q, table, lens, n_new=-1)


def test_keys_of_places_without_a_value():
    """The choice by digits gives places without a value the key 0 and counts them as soon as the
    wanted prefix is 0 after a first digit: none of a value's keys then shares their next digit."""
    lowest = [-math.inf, -3.4028235e38, -3.0e38, -1.8e38, -1.7014118e38, -1.7e38, -8.5e37, -1.0, -1e-38, 0.0, 1.0]
    u = torch.tensor(lowest).view(torch.int32).long() & 0xFFFFFFFF
    keys = torch.where(u >> 31 == 1, ~u & 0xFFFFFFFF, u | 0x80000000).tolist()
    assert keys[0] == 0x007FFFFF and keys == sorted(keys)
    least = keys[0]
    for bits in range(1, 33):                     # of the first pass: the highest in which keys differ
        shift = max(bits - 8, 0)
        if least >> shift == 0:                   # a prefix of 0 is possible
            after = max(shift - 8, 0)
            assert shift < 32 and all((k >> after) & ((1 << (shift - after)) - 1) > 0 for k in keys if k >> shift == 0)


def test_take():
    nan = math.nan
    assert O.take([1, 5, 5, 2], 2, 0, 0) == [1, 2]
    assert O.take([5, 5, 5, 5], 2, 0, 0) == [0, 1]
    assert O.take([9, 1, 2, nan, 0], 3, 1, 1) == [0, 3, 4]
    assert O.take([-0.0, 0.0, -1.0], 1, 0, 0) == [0]
    assert O.take([1, 2], 5, 1, 1) == [0, 1]


def test_scores_bound_every_key():
    """No key of a page scores higher than the page."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 4, 5, 32, generator=g).to(torch.bfloat16)
    k = torch.randn(3, 2, 16, 32, generator=g).to(torch.bfloat16)
    table, lens = torch.tensor([[2, 0, 1]], dtype=torch.int32), [45]
    bnd = O.bounds(k, torch.zeros(3, 2, 2, 32, dtype=torch.bfloat16), table, lens, None)
    s, _ = O.scores(q, bnd, table, lens, None, 16, 0.5, "none")
    for h in range(2):
        keys = O.rows(k, table[0], 45)[h]
        true = 0.5 * (q[0, 2 * h:2 * h + 2].double() @ keys.T).amax(0)      # [Nq, tokens]
        for x in range(3):
            assert bool((true[:, 16 * x:16 * x + 16].amax(1) <= s[0, h, :, x] + 1e-9).all())


def test_weights_of_one_row_sum_to_one():
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(*s, generator=g).to(torch.bfloat16) for s in ((1, 1, 1, 32), (2, 1, 16, 32)))
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    lse = torch.logsumexp(0.2 * (O.rows(k, table[0], 27)[0] @ q[0, 0, 0].double()), 0).reshape(1, 1, 1)
    w, _ = O.weights(q, k, table, [27], lse, torch.zeros(2, 1, 16), None, 0.2, "causal_br", 1.0)
    assert abs(float(w.sum()) - 1) < 1e-9
