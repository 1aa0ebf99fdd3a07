"""CPU: refusals of the norm, append and paged entry points (host checks, before any
CUDA call), and the gradient formula that the kernels are held to against differences."""
import ctypes

import pytest
import torch

from exact_attention_69_gb300 import _lib
from tests import cache_oracle as O

INV, UNS, MIS = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_UNSUPPORTED, _lib.ATTN_ERR_MISALIGNED
A = 1 << 20  # a pointer that no call may touch


@pytest.fixture(scope="module")
def lib():
    from exact_attention_69_gb300 import build
    build.build()
    return _lib.load()


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def test_formula_against_differences():
    """The gradient formula that the kernel is held to, against central differences of
    the definition in 64 bits (step 2^-20, so errors of about 2^-36 of the curvature)."""
    x, w, dy = rnd(21, 1, 2, 3, 32).double(), rnd(22, 32).double(), rnd(23, 1, 2, 3, 32).double()
    pos, freqs = torch.arange(3)[None] + 9, 10000.0 ** (-torch.arange(8, dtype=torch.float64) / 8)
    for il in (False, True):
        dx, _, dw, _ = O.norm_rope_back(x, w, dy, pos, freqs, il, 1e-3)
        f = lambda a, b: float((O.norm_rope(a, b, pos, freqs, il, 1e-3)[0] * dy).sum())  # noqa: E731
        h = 2.0 ** -20
        for at in ((0, 0, 0, 0), (0, 1, 2, 9), (0, 0, 1, 31), (0, 1, 0, 17)):
            e = torch.zeros_like(x)
            e[at] = h
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx[at])) < 1e-7
        for at in (0, 9, 31):
            e = torch.zeros_like(w)
            e[at] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[at])) < 1e-7


def rope():
    p = _lib.AttnRopeParams()
    p.q = p.k = p.q_out = p.k_out = p.inv_freq = A
    p.B, p.N, p.Hq, p.Hk, p.d, p.rot, p.norm, p.eps = 2, 8, 4, 2, 64, 64, 1, 1e-6
    return p


def append():
    p = rope()
    p.k_out = None
    p.v = p.k_cache = p.v_cache = p.block_table = p.starts = A
    p.n_pages, p.page_size, p.table_width, p.table_stride = 9, 16, 4, 4
    return p


def rope_bwd():
    p = _lib.AttnRopeBwdParams()
    for n in ("q", "k", "dq_out", "dk_out", "dq", "dk", "inv_freq"):
        setattr(p, n, A)
    p.B, p.N, p.Hq, p.Hk, p.d, p.rot, p.norm, p.eps = 2, 8, 4, 2, 64, 64, 1, 1e-6
    return p


def paged():
    p = _lib.AttnPagedParams()
    for n in ("q", "k_cache", "v_cache", "o", "block_table", "kv_lens", "prefix_table", "workspace"):
        setattr(p, n, A)
    p.B, p.Hq, p.Hk, p.Nq, p.d, p.scale, p.mask_kind = 2, 8, 2, 1, 64, 0.125, _lib.ATTN_MASK_CAUSAL_BR
    p.n_pages, p.page_size, p.table_width, p.table_stride, p.prefix_len, p.prefix_pages = 9, 16, 4, 4, 20, 2
    p.workspace_bytes = 1 << 40
    return p


BAD_ROPE = [
    (dict(B=0), INV), (dict(N=0), INV), (dict(Hq=0, Hk=0), INV), (dict(Hq=-1), INV), (dict(d=48), UNS),
    (dict(d=256), UNS), (dict(rot=8), INV), (dict(rot=80), INV), (dict(rot=0), INV), (dict(inv_freq=None), INV),
    (dict(inv_freq=A + 4), MIS), (dict(eps=float("nan")), INV), (dict(eps=-1.0), INV),
    (dict(norm=0, q_weight=A), INV), (dict(q_weight=A, q_weight_type=2), INV),
    (dict(k_weight=A + 2, k_weight_type=1), MIS), (dict(positions=A), INV), (dict(pos_type=1), INV),
    (dict(positions=A, pos_type=3), INV), (dict(positions=A + 4, pos_type=2), MIS), (dict(q=None), INV),
    (dict(k=A + 8), MIS), (dict(B=1 << 20, N=1 << 10), INV), (dict(q_stride=(4096, 512, 60)), MIS),
    (dict(q_stride=(4096, -512, 64)), INV), (dict(Hk=0), INV), (dict(Hq=0), INV),
]
BAD_FWD = [(dict(k_out=None), INV), (dict(v=A), INV), (dict(starts=A), INV), (dict(k_out_stride=(1024, 0, 64)), INV),
           (dict(q_out=A + 2), MIS), (dict(q_out_stride=(2048, 512, 32)), INV)]
BAD_APPEND = [(dict(k_out=A), INV), (dict(v=None), INV), (dict(n_pages=0), INV), (dict(page_size=8), INV),
              (dict(page_size=48), INV), (dict(k_cache=None), INV), (dict(v_cache=A + 4), MIS),
              (dict(k_cache_stride=(2048, 0, 64)), INV), (dict(block_table=None), INV), (dict(starts=None), INV),
              (dict(counts=A + 2), MIS), (dict(table_width=0), INV), (dict(table_stride=3), INV)]
BAD_BWD = [(dict(dq=None), INV), (dict(dk_out=A + 2), MIS), (dict(norm=0, dq_weight=A), INV),
           (dict(dk_stride=(1024, 512, 32)), INV), (dict(workspace=A + 8), MIS),
           (dict(q_weight=A, q_weight_type=1, dq_weight=A + 2), MIS)]
BAD_PAGED = [
    (dict(B=0), INV), (dict(Nq=0), INV), (dict(Hk=3), INV), (dict(d=96), UNS), (dict(prefix_len=-1), INV),
    (dict(num_ctas=-1), INV), (dict(scale=0.0), INV), (dict(scale=float("inf")), INV),
    (dict(mask_kind=_lib.ATTN_MASK_CAUSAL), INV), (dict(mask_kind=_lib.ATTN_MASK_NA2D), INV), (dict(inject=2), INV),
    (dict(n_pages=0), INV), (dict(page_size=24), INV), (dict(q=None), INV), (dict(o=A + 8), MIS),
    (dict(o_stride=(512, 0, 64)), INV), (dict(k_cache_stride=(2048, 60, 64)), MIS), (dict(block_table=None), INV),
    (dict(kv_lens=None), INV), (dict(kv_lens=A + 1), MIS), (dict(lse=A + 2), MIS), (dict(table_width=0), INV),
    (dict(table_stride=2), INV), (dict(prefix_len=33), INV), (dict(prefix_table=None), INV),
    (dict(workspace=A + 4), MIS), (dict(table_width=1 << 27, table_stride=1 << 27), INV),
    (dict(B=1 << 20, Nq=1 << 10), INV), (dict(B=1 << 16, Hq=2, table_width=1 << 20, table_stride=1 << 20), INV),
]


def refuses(lib, call, p, changes, code):
    for k, v in changes.items():
        if isinstance(v, tuple):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    assert getattr(lib, call)(ctypes.byref(p)) == code, lib.attn_last_error()
    assert lib.attn_last_error()


@pytest.mark.parametrize("changes,code", BAD_ROPE + BAD_FWD, ids=str)
def test_forward_refuses(lib, changes, code):
    refuses(lib, "attn_qk_norm_rope", rope(), changes, code)


@pytest.mark.parametrize("changes,code", BAD_ROPE + BAD_APPEND, ids=str)
def test_append_refuses(lib, changes, code):
    refuses(lib, "attn_kv_append", append(), changes, code)


@pytest.mark.parametrize("changes,code", [b for b in BAD_ROPE if b[0] not in (dict(Hk=0), dict(Hq=0))] + BAD_BWD, ids=str)
def test_backward_refuses(lib, changes, code):
    refuses(lib, "attn_qk_norm_rope_bwd", rope_bwd(), changes, code)


@pytest.mark.parametrize("changes,code", BAD_PAGED, ids=str)
def test_paged_refuses(lib, changes, code):
    refuses(lib, "attn_paged", paged(), changes, code)


def test_null_blocks(lib):
    for name in ("attn_qk_norm_rope", "attn_kv_append", "attn_qk_norm_rope_bwd", "attn_paged"):
        assert getattr(lib, name)(None) == INV
    for name in ("attn_qk_norm_rope_bwd_workspace_bytes", "attn_paged_workspace_bytes"):
        assert getattr(lib, name)(None) == -INV


def test_python_refuses_cpu_tensors_and_types():
    import exact_attention_69_gb300 as E
    q = torch.zeros(1, 2, 3, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        E.qk_norm_rope_fwd(q, q)
    with pytest.raises(TypeError, match="bfloat16"):
        E.qk_norm_rope_fwd(q.float(), q)
    with pytest.raises(ValueError):
        E.kv_append(q, q, q, q, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="mask"):
        E.attn_paged(q, q, q, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), mask="causal")
    with pytest.raises(ValueError):
        E.rope_freqs(24)


def test_python_refuses_numbers_that_do_not_fit():
    """A number that the library's fields cannot hold is refused, not cut to its low bits."""
    import exact_attention_69_gb300 as E
    q = torch.zeros(1, 2, 3, 32, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for name, bad in (("prefix_len", 2 ** 32 + 5), ("prefix_len", 2 ** 31), ("prefix_len", -2 ** 32), ("num_ctas", 2 ** 32 + 1),
                      ("inject", 2 ** 32), ("timeout_ns", 2 ** 64 + 1), ("timeout_ns", -1)):
        with pytest.raises(ValueError, match=name):
            E.attn_paged(q, q, q, table, lens, **{name: bad})
    from exact_attention_69_gb300 import cache
    with pytest.raises(ValueError, match="a size of q"):
        cache._heads("q", torch.zeros(1, 1, 1, 32, dtype=torch.bfloat16).expand(2 ** 32 + 1, 1, 1, 32))
    with pytest.raises(ValueError, match="a size of table"):
        cache._int32("table", lens.expand(2 ** 31)[:, None], torch.device("cpu"), (None, 1))
    for ok, bits in ((2 ** 31 - 1, 32), (-2 ** 31, 32), (2 ** 63 - 1, 64)):
        assert cache._fits("x", ok, bits) == ok


# strides (b, h, n) under which places of a written tensor lie on one another; B 2, N 8, d 64, 9 pages of 16
OVERLAPS = [
    ("attn_qk_norm_rope", rope, dict(q_out_stride=(64, 64, 64))), ("attn_qk_norm_rope", rope, dict(q_out_stride=(2048, 256, 64))),
    ("attn_qk_norm_rope", rope, dict(k_out_stride=(512, 512, 64))), ("attn_qk_norm_rope", rope, dict(k_out_stride=(64, 128, 128))),
    ("attn_qk_norm_rope", rope, dict(q_out_stride=(1 << 62, 512, 1 << 61))),
    ("attn_kv_append", append, dict(q_out_stride=(1024, 512, 64))), ("attn_kv_append", append, dict(k_cache_stride=(1024, 1024, 64))),
    ("attn_kv_append", append, dict(v_cache_stride=(64, 1024, 64))),
    ("attn_qk_norm_rope_bwd", rope_bwd, dict(dq_stride=(2040, 512, 64))), ("attn_qk_norm_rope_bwd", rope_bwd, dict(dk_stride=(64, 64, 128))),
    ("attn_paged", paged, dict(o_stride=(64, 64, 0))),
]


@pytest.mark.parametrize("call,make,changes", OVERLAPS, ids=lambda x: str(x) if isinstance(x, dict) else None)
def test_written_tensors_that_overlap_themselves(lib, call, make, changes):
    refuses(lib, call, make(), changes, INV)


def test_written_strides_that_do_not_overlap(lib):
    """Heads last, padded rows, any order of the dimensions: the host's checks reach the last
    one that follows (no workspace), or the missing GPU."""
    for st in ((2048, 64, 256), (4096, 512, 64), (64, 128, 512), (2048, 512, 64), (1 << 30, 72, 576)):
        p = rope_bwd()
        p.dq_stride[:] = st
        p.q_weight = p.dq_weight = A
        code = lib.attn_qk_norm_rope_bwd(ctypes.byref(p))
        said = lib.attn_last_error()
        assert b"overlap" not in said and (code != INV or b"workspace" in said), said
