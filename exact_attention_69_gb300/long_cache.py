"""Python entry points that keep a long paged cache affordable, over libattn.so.

    kv_bounds(k_cache, ...)       lower and upper bounds of every channel of a page's keys
    block_scores(q, bounds, ...)  the largest score that a key of each page can have
    block_select(scores, ...)     the pages that each query reads
    attn_blocks(q, k_cache, ...)  attention over the selected pages
    kv_weights(q, k_cache, ...)   the attention weight that every cached token received
    kv_evict(k_cache, ...)        the cache cut to a budget, by those weights

Layouts are those of attn_paged and kv_append: q [B, Hq, Nq, d] bf16 with any strides
whose last dimension is contiguous; a cache [n_pages, Hk, page_size, d] bf16; tables,
lengths and lists int32 on the device. The queries of sequence b are the last q_lens[b]
(None: Nq) of its kv_lens[b] tokens; mask 'causal_br': query i sees slots up to i +
kv_lens[b] - q_lens[b]; 'none': all of them. Page x of a sequence is entry x of its row
in the block table; a prefix that sequences share is pages that several rows name, for
the calls that read them: pages that kv_weights or kv_evict writes must be one
sequence's only (what to do with a shared prefix is said there).

A decoding step over a long cache:

    q = kv_append(...)                                    # the new token
    kv_bounds(k_cache, bounds, table, lens, n_new=1)      # its page's bounds
    scores = block_scores(q, bounds, table, lens, page_size=page)
    pages = block_select(scores, lens, 32, page_size=page)
    o = attn_blocks(q, k_cache, v_cache, table, lens, pages, return_lse=False)

Keeping a cache within a budget: kv_weights after each attn_paged, with its lse, and
kv_evict when a sequence has grown too long. No gradient goes through any of them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from .cache import _PAGED_MASKS, _fits, _heads, _int32, _on, _plans, _ptr, _remember, _same_device, _sig, _wrote

_Params, _byref, _empty = _lib.AttnLongParams, ctypes.byref, torch.empty
_device_now, _stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _plain(name, t, dtype, device, shape):
    """Checks a contiguous tensor of the library's own layout."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _mask(mask):
    if mask not in _PAGED_MASKS:
        raise ValueError(f"mask must be 'none' or 'causal_br', not {mask!r}")
    return _PAGED_MASKS[mask]


def _pages(p, name, cache):
    if cache.dim() != 4:
        raise ValueError(f"{name} must be [n_pages, Hk, page_size, d]")
    p.n_pages, p.Hk, p.page_size, p.d = cache.shape
    for n in cache.shape:
        _fits(f"a size of {name}", n)


def _tables(p, device, block_table, kv_lens, q_lens=None):
    if block_table is not None:
        _int32("block_table", block_table, device, (None, None))
        p.B, p.table_width = block_table.shape
        p.table_stride = block_table.stride(0)
    _int32("kv_lens", kv_lens, device, (p.B,))
    if q_lens is not None:
        _int32("q_lens", q_lens, device, (p.B,))


def _queries(p, q, device, mask, scale):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    p.q_stride[:] = _heads("q", q, (p.B, q.shape[1], q.shape[2], p.d))
    _same_device(device, q=q)
    p.Hq, p.Nq = q.shape[1], q.shape[2]
    p.mask_kind = _mask(mask)
    p.scale = float(1.0 / math.sqrt(p.d) if scale is None else scale)


_calls: dict = {}


def _call(name, p):
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(_lib.load(), name)
    code = f(_byref(p))
    if code:
        _lib.check(code, name.replace("attn_kv", "kv").replace("attn_block_", "block_"))


# A call on the current stream of the current device, the usual one, goes straight to
# its _run_ function; others go there through _on.


def _form(p, full_tiles, timeout_ns, inject):
    """The fields of the calls that have a form with tiles of 128 rows."""
    if timeout_ns < 0:
        raise ValueError("timeout_ns must be >= 0")
    p.full_tiles = 0 if full_tiles is None else 1 if full_tiles else 2
    p.timeout_ns, p.inject = _fits("timeout_ns", timeout_ns, 64), _fits("inject", inject)


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _plan_bounds(k_cache, bounds, block_table, kv_lens):
    p = _Params()
    _pages(p, "k_cache", k_cache)
    p.k_cache_stride[:] = _heads("k_cache", k_cache)
    device = k_cache.device
    _tables(p, device, block_table, kv_lens)
    _plain("bounds", bounds, torch.bfloat16, device, (p.n_pages, p.Hk, 2, p.d))
    return bytes(p)


def kv_bounds(k_cache: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor, *,
              n_new: int | None = None, stream=None) -> None:
    """Brings the bounds of the pages' keys up to date, in place.

    bounds [n_pages, Hk, 2, d] bf16: the least (0) and the greatest (1) value of every
    channel over the page's slots below the sequence's end. Pages that hold one of the
    newest `n_new` tokens of each sequence (kv_lens [B] counts them in) are looked at,
    each whole; None: every page that holds a token. Exact; NaN keys give NaN bounds.
    Sequences may share pages that are full in each.
    """
    if n_new is not None and int(n_new) < 0:
        raise ValueError("n_new must be >= 0")
    n_new = -1 if n_new is None else _fits("n_new", int(n_new))
    key = ("bounds", _sig(k_cache), _sig(bounds), _sig(block_table), _sig(kv_lens))
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_bounds(k_cache, bounds, block_table, kv_lens))
    p = _Params.from_buffer_copy(plan)
    p.k_cache, p.bounds, p.block_table, p.kv_lens = k_cache.data_ptr(), bounds.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr()
    p.n_new = n_new
    device = k_cache.device
    if stream is None and _device_now() == device.index:
        return _run_bounds(_stream_now(device.index), p, bounds)
    _on(device, stream, (k_cache, bounds, block_table, kv_lens), lambda handle: _run_bounds(handle, p, bounds))


def _run_bounds(handle, p, bounds):
    p.stream = handle
    _call("attn_kv_bounds", p)
    _wrote((bounds,))


def _plan_scores(q, bounds, block_table, kv_lens, page_size, q_lens, scale, mask, out, full_tiles, timeout_ns, inject):
    p = _Params()
    _fits("page_size", page_size)
    _form(p, full_tiles, timeout_ns, inject)
    device = _cuda(bounds, "bounds")
    if bounds.dim() != 4:
        raise ValueError("bounds must be [n_pages, Hk, 2, d]")
    p.n_pages, p.Hk, _, p.d = bounds.shape
    p.page_size = page_size
    _plain("bounds", bounds, torch.bfloat16, device, (p.n_pages, p.Hk, 2, p.d))
    _tables(p, device, block_table, kv_lens, q_lens)
    _queries(p, q, device, mask, scale)
    if out is not None:
        _plain("out", out, torch.float32, device, (p.B, p.Hk, p.Nq, p.table_width))
    return bytes(p), (p.B, p.Hk, p.Nq, p.table_width)


def block_scores(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor, *,
                 page_size: int, q_lens: torch.Tensor | None = None, scale: float | None = None,
                 mask: str = "causal_br", out: torch.Tensor | None = None, full_tiles: bool | None = None,
                 timeout_ns: int = 0, inject: int = 0, stream=None) -> torch.Tensor:
    """How large a score each page's keys can have with each query, from kv_bounds.

    Returns fp32 [B, Hk, Nq, width of the table]: the largest over the query heads of a
    key head of scale * sum_c (min(q_c, 0) lower_c + max(q_c, 0) upper_c), -inf for pages
    of which the query sees nothing. scale None: 1 / sqrt(d). full_tiles, timeout_ns and
    inject: as attn_blocks has them, but the form for few rows holds 32 (Nq times the
    query heads of a key head, those rounded up to 4 or a multiple of 8): False with more
    is refused.
    """
    page_size, timeout_ns, inject = int(page_size), int(timeout_ns), int(inject)
    scale = None if scale is None else float(scale)
    full_tiles = None if full_tiles is None else bool(full_tiles)
    key = ("scores", _sig(q), _sig(bounds), _sig(block_table), _sig(kv_lens), page_size, _sig(q_lens), scale, mask,
           _sig(out), full_tiles, timeout_ns, inject)
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_scores(q, bounds, block_table, kv_lens, page_size, q_lens, scale, mask, out, full_tiles,
                                           timeout_ns, inject))
    p = _Params.from_buffer_copy(plan[0])
    p.q, p.bounds, p.block_table, p.kv_lens = q.data_ptr(), bounds.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr()
    p.q_lens = _ptr(q_lens)
    device = q.device
    if stream is None and _device_now() == device.index:
        return _run_scores(_stream_now(device.index), p, plan[1], device, out)
    return _on(device, stream, (q, bounds, block_table, kv_lens, q_lens, out),
               lambda handle: _run_scores(handle, p, plan[1], device, out))


def _run_scores(handle, p, shape, device, out):
    s = _empty(shape, dtype=torch.float32, device=device) if out is None else out
    p.scores, p.stream = s.data_ptr(), handle
    _call("attn_block_scores", p)
    if out is not None:
        _wrote((out,))
    return s


def _plan_select(scores, kv_lens, n, page_size, q_lens, first, last, mask, out):
    p = _Params()
    for name, x in (("n", n), ("page_size", page_size), ("first", first), ("last", last)):
        _fits(name, x)
    if n < 1 or first < 0 or last < 0 or first + last > n:
        raise ValueError("n must be >= 1, first and last >= 0 and no more than n together")
    device = _cuda(scores, "scores")
    if scores.dim() != 4:
        raise ValueError("scores must be [B, Hk, Nq, pages]")
    _plain("scores", scores, torch.float32, device, scores.shape)
    for x in scores.shape:
        _fits("a size of scores", x)
    p.B, p.Hk, p.Nq, p.table_width = scores.shape
    p.page_size, p.n, p.first, p.last, p.mask_kind = page_size, n, first, last, _mask(mask)
    _tables(p, device, None, kv_lens, q_lens)
    if out is not None:
        _plain("out", out, torch.int32, device, (p.B, p.Hk, p.Nq, n))
    return bytes(p), (p.B, p.Hk, p.Nq, n)


def block_select(scores: torch.Tensor, kv_lens: torch.Tensor, n: int, *, page_size: int,
                 q_lens: torch.Tensor | None = None, first: int = 1, last: int = 2, mask: str = "causal_br",
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The pages that each query reads: int32 [B, Hk, Nq, n], ascending, -1 behind the last.

    Of the pages that the query sees the `first` first and the `last` last ones and those
    of the greatest score (scores [B, Hk, Nq, pages], block_scores) among the others, n in
    all; every one if it sees no more. Ties go to the lowest page, NaN counts as the
    greatest score.
    """
    n, page_size, first, last = int(n), int(page_size), int(first), int(last)
    key = ("select", _sig(scores), _sig(kv_lens), n, page_size, _sig(q_lens), first, last, mask, _sig(out))
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_select(scores, kv_lens, n, page_size, q_lens, first, last, mask, out))
    p = _Params.from_buffer_copy(plan[0])
    p.scores, p.kv_lens, p.q_lens = scores.data_ptr(), kv_lens.data_ptr(), _ptr(q_lens)
    device = scores.device
    if stream is None and _device_now() == device.index:
        return _run_select(_stream_now(device.index), p, plan[1], device, out)
    return _on(device, stream, (scores, kv_lens, q_lens, out), lambda handle: _run_select(handle, p, plan[1], device, out))


def _run_select(handle, p, shape, device, out):
    blocks = _empty(shape, dtype=torch.int32, device=device) if out is None else out
    p.blocks, p.stream = blocks.data_ptr(), handle
    _call("attn_block_select", p)
    if out is not None:
        _wrote((out,))
    return blocks


def _plan_blocks(q, k_cache, v_cache, block_table, kv_lens, blocks, q_lens, scale, mask, out, lse, full_tiles,
                 timeout_ns, inject):
    p = _Params()
    _form(p, full_tiles, timeout_ns, inject)
    _pages(p, "k_cache", k_cache)
    p.k_cache_stride[:] = _heads("k_cache", k_cache)
    p.v_cache_stride[:] = _heads("v_cache", v_cache, k_cache.shape)
    device = k_cache.device
    _same_device(device, v_cache=v_cache, out=out, lse=lse)
    _tables(p, device, block_table, kv_lens, q_lens)
    _queries(p, q, device, mask, scale)
    if blocks.dim() != 4:
        raise ValueError("blocks must be [B, Hk, Nq, n]")
    _plain("blocks", blocks, torch.int32, device, (p.B, p.Hk, p.Nq, blocks.shape[3]))
    p.n = _fits("a size of blocks", blocks.shape[3])
    if out is not None:
        p.o_stride[:] = _heads("out", out, q.shape)
    if lse is not None:
        _plain("lse", lse, torch.float32, device, q.shape[:3])
    return bytes(p)


def attn_blocks(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                kv_lens: torch.Tensor, blocks: torch.Tensor, *, q_lens: torch.Tensor | None = None,
                scale: float | None = None, mask: str = "causal_br", out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, return_lse: bool = True, full_tiles: bool | None = None,
                timeout_ns: int = 0, inject: int = 0, stream=None):
    """Attention of each query over the pages that it selected.

    As attn_paged over the whole cache, but query i of a key head's query heads sees only
    slots of the pages in blocks[b, h, i] (block_select, or any list: entries of the
    sequence's row in the block table, in any order; a page named twice counts once,
    negative entries and pages of which the query sees nothing not at all). A row without
    a slot gives 0 and an LSE of -inf. Values of slots that only some queries of a
    sequence read must be finite. full_tiles: None for the library's choice by sizes, True
    for tiles of 128 rows, False for the form for few rows, which takes more time for many
    rows and is the finer one (softmax weights enter the second product as two bf16 parts
    there, as one in the tiles: O is off by 0.0017 and 0.0023 of its norm, of which its own
    rounding is 0.0017); timeout_ns: bound on every wait on the device (0: two seconds;
    device_status says if one ran out); inject: test hook.

    Returns (o, lse) or o; no gradient goes through it.
    """
    scale, timeout_ns, inject = None if scale is None else float(scale), int(timeout_ns), int(inject)
    full_tiles = None if full_tiles is None else bool(full_tiles)
    key = ("blocks", _sig(q), _sig(k_cache), _sig(v_cache), _sig(block_table), _sig(kv_lens), _sig(blocks),
           _sig(q_lens), scale, mask, _sig(out), _sig(lse), full_tiles, timeout_ns, inject)
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_blocks(q, k_cache, v_cache, block_table, kv_lens, blocks, q_lens, scale, mask, out,
                                           lse, full_tiles, timeout_ns, inject))
    p = _Params.from_buffer_copy(plan)
    p.q, p.k_cache, p.v_cache, p.block_table = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr()
    p.kv_lens, p.q_lens, p.blocks = kv_lens.data_ptr(), _ptr(q_lens), blocks.data_ptr()
    device = q.device
    if stream is None and _device_now() == device.index:
        return _run_blocks(_stream_now(device.index), p, q.shape, device, out, lse, return_lse)
    return _on(device, stream, (q, k_cache, v_cache, block_table, kv_lens, blocks, q_lens, out, lse),
               lambda handle: _run_blocks(handle, p, q.shape, device, out, lse, return_lse))


def _run_blocks(handle, p, shape, device, out, lse, return_lse):
    o = _empty(shape, dtype=torch.bfloat16, device=device) if out is None else out
    z = _empty(shape[:3], dtype=torch.float32, device=device) if lse is None and return_lse else lse
    p.o, p.lse, p.stream = o.data_ptr(), _ptr(z), handle
    _call("attn_blocks", p)
    if out is not None or lse is not None:
        _wrote([t for t in (out, lse) if t is not None])
    return (o, z) if return_lse else o


def _plan_weights(q, k_cache, block_table, kv_lens, lse, weights, q_lens, scale, mask, decay, out, full_tiles, timeout_ns,
                  inject):
    p = _Params()
    if not (math.isfinite(decay) and decay >= 0):
        raise ValueError("decay must be finite and >= 0")
    _form(p, full_tiles, timeout_ns, inject)
    _pages(p, "k_cache", k_cache)
    p.k_cache_stride[:] = _heads("k_cache", k_cache)
    device = k_cache.device
    _tables(p, device, block_table, kv_lens, q_lens)
    _queries(p, q, device, mask, scale)
    _plain("lse", lse, torch.float32, device, q.shape[:3])
    for name, t in (("weights", weights), ("out", out)):
        if t is not None:
            _plain(name, t, torch.float32, device, (p.n_pages, p.Hk, p.page_size))
    p.decay = decay
    return bytes(p)


def kv_weights(q: torch.Tensor, k_cache: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
               lse: torch.Tensor, weights: torch.Tensor, *, q_lens: torch.Tensor | None = None, decay: float = 1.0,
               scale: float | None = None, mask: str = "causal_br", out: torch.Tensor | None = None,
               full_tiles: bool | None = None, timeout_ns: int = 0, inject: int = 0, stream=None) -> None:
    """Adds the attention that cached tokens received from these queries to their weights.

    weights [n_pages, Hk, page_size] fp32, in place (or into `out`, for the slots that the
    sequences hold): decay * weights + the sum over the queries that see the slot and the
    query heads of its key head of exp(scale * q . k - lse), with the lse [B, Hq, Nq] that
    attn_paged (a shared prefix counted in) or attn_blocks returned for the same queries.
    With 'causal_br' the queries' own slots are new and start from zero, whatever a
    recycled page held; with decay 0 all slots do. Sums are fp32 in a fixed order.
    No page may be in two rows of the table: each sequence reads, adds to and writes its
    pages' weights, and one's sums would be lost. With a prefix that sequences share,
    multiply `weights` by the decay, then call once for each sequence (its rows of q,
    block_table, kv_lens, q_lens and lse), with decay 1, on one stream.
    full_tiles, timeout_ns and inject: as attn_blocks has them, but the form for few rows
    holds 32 (Nq times the query heads of a key head): False with more is refused.
    """
    decay, timeout_ns, inject = float(decay), int(timeout_ns), int(inject)
    scale = None if scale is None else float(scale)
    full_tiles = None if full_tiles is None else bool(full_tiles)
    key = ("weights", _sig(q), _sig(k_cache), _sig(block_table), _sig(kv_lens), _sig(lse), _sig(weights), _sig(q_lens),
           scale, mask, decay, _sig(out), full_tiles, timeout_ns, inject)
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_weights(q, k_cache, block_table, kv_lens, lse, weights, q_lens, scale, mask, decay,
                                            out, full_tiles, timeout_ns, inject))
    p = _Params.from_buffer_copy(plan)
    p.q, p.k_cache, p.block_table, p.kv_lens = q.data_ptr(), k_cache.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr()
    p.lse, p.weights, p.q_lens = lse.data_ptr(), weights.data_ptr(), _ptr(q_lens)
    to = weights if out is None else out
    p.weights_out = to.data_ptr()
    device = q.device
    if stream is None and _device_now() == device.index:
        return _run_weights(_stream_now(device.index), p, to)
    _on(device, stream, (q, k_cache, block_table, kv_lens, lse, weights, q_lens, out), lambda handle: _run_weights(handle, p, to))


def _run_weights(handle, p, to):
    p.stream = handle
    _call("attn_kv_weights", p)
    _wrote((to,))


def _plan_evict(k_cache, v_cache, weights, block_table, kv_lens, budget, first, last, dst_table):
    p = _Params()
    for name, x in (("budget", budget), ("first", first), ("last", last)):
        _fits(name, x)
    if budget < 1 or first < 0 or last < 0 or first + last > budget:
        raise ValueError("budget must be >= 1, first and last >= 0 and no more than budget together")
    _pages(p, "k_cache", k_cache)
    p.k_cache_stride[:] = _heads("k_cache", k_cache)
    p.v_cache_stride[:] = _heads("v_cache", v_cache, k_cache.shape)
    device = k_cache.device
    _same_device(device, v_cache=v_cache)
    _plain("weights", weights, torch.float32, device, (p.n_pages, p.Hk, p.page_size))
    _tables(p, device, block_table, kv_lens)
    if dst_table is not None:
        _int32("dst_table", dst_table, device, (p.B, None))
        p.dst_width, p.dst_stride = dst_table.shape[1], dst_table.stride(0)
    p.n, p.first, p.last = budget, first, last
    return bytes(p), p.B, p.Hk


def kv_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, block_table: torch.Tensor,
             kv_lens: torch.Tensor, budget: int, *, first: int = 0, last: int = 0,
             dst_table: torch.Tensor | None = None, stream=None):
    """Cuts every sequence's cache to `budget` tokens for each key head, in place.

    Kept are the `first` first and the `last` last tokens and those of the greatest weight
    (kv_weights) among the others, ties to the earliest, NaN as the greatest; every token
    if there are no more. Their keys, values and weights move, in their order, to the
    front of the sequence's pages, or to the pages of dst_table [B, width] (a copy; none
    of them may be in block_table). Pages that are written must be one sequence's only:
    in place, no page may be in two rows of block_table; sequences that share a prefix
    are cut into pages of dst_table, each of which is in it once. Returns (new_lens [B],
    kept [B, Hk, budget]): the lengths after it and the slots that the tokens came from,
    -1 behind the last. Key heads keep different tokens: give kv_append the tokens' true
    positions from then on, and find the pages' bounds again (kv_bounds) where they are used.
    """
    budget, first, last = int(budget), int(first), int(last)
    key = ("evict", _sig(k_cache), _sig(v_cache), _sig(weights), _sig(block_table), _sig(kv_lens), budget, first, last,
           _sig(dst_table))
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_evict(k_cache, v_cache, weights, block_table, kv_lens, budget, first, last,
                                          dst_table))
    p = _Params.from_buffer_copy(plan[0])
    p.k_cache, p.v_cache, p.weights = k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr()
    p.block_table, p.kv_lens, p.dst_table = block_table.data_ptr(), kv_lens.data_ptr(), _ptr(dst_table)
    device = k_cache.device
    if stream is None and _device_now() == device.index:
        return _run_evict(_stream_now(device.index), p, plan, device, k_cache, v_cache, weights)
    return _on(device, stream, (k_cache, v_cache, weights, block_table, kv_lens, dst_table),
               lambda handle: _run_evict(handle, p, plan, device, k_cache, v_cache, weights))


def _run_evict(handle, p, plan, device, k_cache, v_cache, weights):
    lens = _empty(plan[1], dtype=torch.int32, device=device)
    kept = _empty((plan[1], plan[2], p.n), dtype=torch.int32, device=device)
    p.new_lens, p.kept, p.stream = lens.data_ptr(), kept.data_ptr(), handle
    _call("attn_kv_evict", p)
    _wrote((k_cache, v_cache, weights))
    return lens, kept
