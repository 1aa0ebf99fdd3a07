"""Python entry points around the attention of a language model, over libattn.so.

    rope_freqs(rot)                 frequencies of the rotary positions
    qk_norm_rope(q, k, ...)         per-head root-mean-square norm and rotary positions in
                                    one pass; differentiable (qk_norm_rope_fwd, _bwd: its halves)
    kv_append(k, v, k_cache, ...)   new keys and values into their pages, normed and rotated
                                    on the way, the queries of the same tokens beside them
    attn_paged(q, k_cache, ...)     attention over the pages, with a prefix that the whole
                                    batch shares

Layouts are the framework's: q, k, v [B, H, N, d] bf16 with any strides whose last
dimension is contiguous (views of a fused projection are read in place); a cache is
[n_pages, Hk, page_size, d] bf16 (a [n_pages, page_size, Hk, d] one as its transposed
view); tables, lengths, starts and counts are int32 on the device, so a captured graph
follows them. Scratch comes from PyTorch's allocator on the call's stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib

_WEIGHT_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_POS_TYPES = {torch.int32: 1, torch.int64: 2}


def rope_freqs(rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """Radians per position of each rotated pair, base^(-2i / rot), i < rot / 2: the
    float64 tensor that `inv_freq` takes. Scaled variants are tensors of the same shape."""
    if rot <= 0 or rot % 16:
        raise ValueError("rot must be a positive multiple of 16")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)


# Plans: a call's checks and the parts of its parameter block that follow from the
# shapes, strides, types and devices of its tensors and from its options, made once for
# each combination of them and copied for every call; pointers are filled in each time.
_plans: dict = {}


def _remember(key, plan):
    if len(_plans) >= 4096:
        _plans.clear()
    _plans[key] = plan
    return plan


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _fits(name, x, bits=32):
    """x, if a signed field of the library's parameter blocks holds it (ctypes drops what does not fit)."""
    if not -(1 << (bits - 1)) <= x < 1 << (bits - 1):
        raise ValueError(f"{name} ({x}) is not a {bits}-bit number")
    return x


def _heads(name, t, shape=None):
    """Checks a [B, H, N, d] bf16 CUDA tensor; returns its element strides (b, h, n)."""
    for n in t.shape:
        _fits(f"a size of {name}", n)
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    a, b, c, last = t.stride()
    if last != 1:
        raise ValueError(f"the last (head) dimension of {name} must be contiguous")
    if not (a or b or c):  # all-zero strides mean "contiguous" to the library
        if t.shape[:3].numel() > 1:
            raise ValueError(f"{name} is expanded in every dimension")
        return (0, 0, t.shape[3])
    return (a, b, c)


def _int32(name, t, device, shape):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() != len(shape) or any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must have the shape {tuple('any' if s is None else s for s in shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    for n in t.shape:
        _fits(f"a size of {name}", n)


def _same_device(device, **ts):
    for name, t in ts.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")


def _weight(name, w, d, device):
    if w is None:
        return 0
    if w.dtype not in _WEIGHT_TYPES:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if w.device != device:
        raise ValueError(f"{name} must be on {device}")
    if w.shape != (d,) or (d > 1 and w.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous [{d}] tensor")
    return _WEIGHT_TYPES[w.dtype]


def _set_rope(p, B, N, d, device, q_weight, k_weight, inv_freq, positions, interleaved, eps):
    """The fields that the forward's and the backward's plans share."""
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights need a norm: give eps")
    else:
        p.norm, p.eps = 1, eps
    p.q_weight_type = _weight("q_weight", q_weight, d, device)
    p.k_weight_type = _weight("k_weight", k_weight, d, device)
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64:
            raise TypeError("inv_freq must be float64 (rope_freqs)")
        if inv_freq.device != device:
            raise ValueError(f"inv_freq must be on {device}")
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous [rot / 2] tensor")
        p.rot = 2 * inv_freq.shape[0]
        if p.rot == 0:
            raise ValueError("inv_freq must not be empty")
    p.interleaved = int(interleaved)
    if positions is not None:
        if positions.dtype not in _POS_TYPES:
            raise TypeError("positions must be int32 or int64")
        if positions.device != device:
            raise ValueError(f"positions must be on {device}")
        if tuple(positions.shape) not in ((N,), (B, N)):
            raise ValueError(f"positions must be [{N}] or [{B}, {N}]")
        p.pos_type = _POS_TYPES[positions.dtype]
        st = positions.stride()
        p.pos_stride[:] = (0, st[0]) if len(st) == 1 else st


def _wrote(ts):
    """Tells autograd which of the caller's tensors a call has written: a graph that saved one
    refuses its backward pass, as after any in-place op."""
    torch.autograd.graph.increment_version(ts)


def _on(device, stream, tensors, run):
    """run(handle) with the tensors' device and the call's stream current, so that
    outputs and scratch come from that stream's memory. Inputs of a call on another
    stream than the current one are held for it until its work so far is done."""
    if stream is None and torch.cuda.current_device() == device.index:
        return run(torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device):
        if stream is None or stream == torch.cuda.current_stream(device):
            return run(torch.cuda.current_stream(device).cuda_stream)
        if stream.device != device:
            raise ValueError(f"the stream must be on {device}")
        with torch.cuda.stream(stream):
            out = run(stream.cuda_stream)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return out


def _plan_fwd(q, k, q_weight, k_weight, inv_freq, positions, interleaved, eps, q_out, k_out):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, Hq, N, d = q.shape
    p = _lib.AttnRopeParams()
    p.B, p.N, p.Hq, p.d = B, N, Hq, d
    p.q_stride[:] = _heads("q", q)
    if k is not None:
        if k.dim() != 4:
            raise ValueError("expected [B, H, N, d] tensors")
        p.Hk = k.shape[1]
        p.k_stride[:] = _heads("k", k, (B, p.Hk, N, d))
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    _same_device(q.device, k=k, q_out=q_out, k_out=k_out)
    _set_rope(p, B, N, d, q.device, q_weight, k_weight, inv_freq, positions, interleaved, eps)
    if q_out is not None:
        p.q_out_stride[:] = _heads("q_out", q_out, q.shape)
    if k_out is not None:
        p.k_out_stride[:] = _heads("k_out", k_out, k.shape)
    return bytes(p)


def qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, *, inv_freq: torch.Tensor | None = None,
                     positions: torch.Tensor | None = None, position_offset: int = 0,
                     interleaved: bool = False, eps: float | None = 1e-6,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm and rotation of every head of q [B, Hq, N, d] and k [B, Hk, N, d] in one pass.

    Each head is divided by the root of its channels' mean square plus `eps` and
    multiplied by its weight ([d], bf16 or fp32; None = ones); eps None: no norm. Then
    the first 2 * len(inv_freq) channels are rotated (rope_freqs; None: no rotation) by
    the token's position: `positions` [N] or [B, N] int32 or int64, else position_offset
    + n. Pairs are (i, i + rot / 2), or (2i, 2i + 1) with `interleaved`. k may be None.
    Returns (q_out, k_out); q_out may be q, k_out k. No gradient goes through it:
    qk_norm_rope is the differentiable one.
    """
    interleaved, eps = bool(interleaved), None if eps is None else float(eps)
    key = ("fwd", _sig(q), _sig(k), _sig(q_weight), _sig(k_weight), _sig(inv_freq), _sig(positions), _sig(q_out),
           _sig(k_out), interleaved, eps)
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_fwd(q, k, q_weight, k_weight, inv_freq, positions, interleaved, eps, q_out, k_out))
    p = _lib.AttnRopeParams.from_buffer_copy(plan)
    p.q, p.k, p.q_weight, p.k_weight = q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight)
    p.inv_freq, p.positions = _ptr(inv_freq), _ptr(positions)
    p.pos_offset = _fits("position_offset", int(position_offset), 64)

    def run(handle):  # (outputs that are made here are contiguous: strides of zero)
        qo = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if q_out is None else q_out
        p.q_out = qo.data_ptr()
        ko = k_out
        if k is not None:
            if ko is None:
                ko = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device)
            p.k_out = ko.data_ptr()
        p.stream = handle
        code = _lib.load().attn_qk_norm_rope(ctypes.byref(p))
        if code:
            _lib.check(code, "qk_norm_rope")
        if q_out is not None or k_out is not None:
            _wrote([t for t in (q_out, k_out) if t is not None])
        return qo, ko

    return _on(q.device, stream, (q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out), run)


def _plan_bwd(q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, positions, interleaved, eps, weight_grads):
    """(the parameter block, bytes of workspace)"""
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    B, Hq, N, d = q.shape
    p = _lib.AttnRopeBwdParams()
    p.B, p.N, p.Hq, p.d = B, N, Hq, d
    p.q_stride[:] = _heads("q", q)
    p.dq_out_stride[:] = _heads("dq_out", dq_out, q.shape)
    if k is not None:
        if k.dim() != 4:
            raise ValueError("expected [B, H, N, d] tensors")
        p.Hk = k.shape[1]
        p.k_stride[:] = _heads("k", k, (B, p.Hk, N, d))
        p.dk_out_stride[:] = _heads("dk_out", dk_out, k.shape)
    elif k_weight is not None:
        raise ValueError("k_weight needs k")
    _same_device(q.device, k=k, dq_out=dq_out, dk_out=dk_out)
    _set_rope(p, B, N, d, q.device, q_weight, k_weight, inv_freq, positions, interleaved, eps)
    plan, n = bytes(p), 0
    if any(weight_grads):
        p.inv_freq, p.positions = _ptr(inv_freq), _ptr(positions)
        p.q_weight, p.k_weight = _ptr(q_weight), _ptr(k_weight)
        p.dq_weight, p.dk_weight = (_ptr(w) if want else None for w, want in zip((q_weight, k_weight), weight_grads))
        with torch.cuda.device(q.device):
            n = _lib.load().attn_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(p))
        if n < 0:
            _lib.check(int(-n), "qk_norm_rope_bwd")
    return plan, int(n)


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor | None, dq_out: torch.Tensor,
                     dk_out: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, *, inv_freq: torch.Tensor | None = None,
                     positions: torch.Tensor | None = None, position_offset: int = 0,
                     interleaved: bool = False, eps: float | None = 1e-6,
                     weight_grads: bool | tuple[bool, bool] = True, stream=None):
    """Gradients through qk_norm_rope_fwd: (dq, dk, dq_weight, dk_weight) for the
    gradients dq_out, dk_out at its outputs; the other arguments as the forward had them.
    Weight gradients have the weights' types (None without a weight, or where weight_grads,
    one for both or a pair, is False); their sums are fp32 in a fixed order."""
    interleaved, eps = bool(interleaved), None if eps is None else float(eps)
    want_q, want_k = weight_grads if isinstance(weight_grads, (tuple, list)) else (weight_grads, weight_grads)
    weight_grads = (bool(want_q) and q_weight is not None, bool(want_k) and k_weight is not None)
    key = ("bwd", _sig(q), _sig(k), _sig(dq_out), _sig(dk_out), _sig(q_weight), _sig(k_weight), _sig(inv_freq),
           _sig(positions), interleaved, eps, weight_grads)
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_bwd(q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, positions, interleaved, eps,
                                        weight_grads))
    p = _lib.AttnRopeBwdParams.from_buffer_copy(plan[0])
    p.q, p.k, p.dq_out, p.dk_out = q.data_ptr(), _ptr(k), dq_out.data_ptr(), _ptr(dk_out)
    p.q_weight, p.k_weight = _ptr(q_weight), _ptr(k_weight)
    p.inv_freq, p.positions = _ptr(inv_freq), _ptr(positions)
    p.pos_offset = _fits("position_offset", int(position_offset), 64)

    def run(handle):
        dk = dwq = dwk = None
        dq = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        p.dq = dq.data_ptr()
        if k is not None:
            dk = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device)
            p.dk = dk.data_ptr()
        if weight_grads[0]:
            dwq = torch.empty_like(q_weight)
            p.dq_weight = dwq.data_ptr()
        if weight_grads[1]:
            dwk = torch.empty_like(k_weight)
            p.dk_weight = dwk.data_ptr()
        if plan[1]:
            ws = torch.empty(plan[1], dtype=torch.uint8, device=q.device)
            p.workspace, p.workspace_bytes = ws.data_ptr(), plan[1]
        p.stream = handle
        code = _lib.load().attn_qk_norm_rope_bwd(ctypes.byref(p))
        if code:
            _lib.check(code, "qk_norm_rope_bwd")
        return dq, dk, dwq, dwk

    return _on(q.device, stream, (q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, positions), run)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, opts):
        qo, ko = qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq=inv_freq, positions=positions, **opts)
        ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq, positions)
        ctx.opts = opts
        ctx.set_materialize_grads(False)
        return qo, ko

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, inv_freq, positions = ctx.saved_tensors
        how = dict(inv_freq=inv_freq, positions=positions, **ctx.opts)
        need_q, need_k, need_wq, need_wk = ctx.needs_input_grad[:4]
        dq = dk = dwq = dwk = None

        def ready(g):  # most strides will do as they are: see attn_rope_bwd_params
            if g.data_ptr() % 16 == 0 and (g.is_contiguous() or (g.stride(3) == 1 and all(
                    n == 1 or (s > 0 and s % 8 == 0) for s, n in zip(g.stride(), g.shape[:3])))):
                return g
            return g.clone(memory_format=torch.contiguous_format)  # (contiguous() would keep a misaligned one)

        # a side is left out if the loss does not reach its output, or nothing of it needs a gradient
        on_q = dq_out is not None and (need_q or need_wq)
        on_k = dk_out is not None and (need_k or need_wk)
        if on_q and on_k:
            dq, dk, dwq, dwk = qk_norm_rope_bwd(q, k, ready(dq_out), ready(dk_out), q_weight, k_weight,
                                                weight_grads=(need_wq, need_wk), **how)
        elif on_q:
            dq, _, dwq, _ = qk_norm_rope_bwd(q, None, ready(dq_out), None, q_weight, None,
                                             weight_grads=(need_wq, False), **how)
        elif on_k:
            dk, _, dwk, _ = qk_norm_rope_bwd(k, None, ready(dk_out), None, k_weight, None,
                                             weight_grads=(need_wk, False), **how)
        if not need_q:
            dq = None
        if not need_k:
            dk = None
        return dq, dk, dwq, dwk, None, None, None


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, *, inv_freq: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, position_offset: int = 0,
                 interleaved: bool = False, eps: float | None = 1e-6):
    """qk_norm_rope_fwd as a differentiable torch op: gradients for q, k and the weights
    (once: the gradient itself is not differentiable). Runs on the current stream. As for
    any PyTorch op, a backward pass is captured into a graph only while no eager graph
    of the same leaves is alive."""
    opts = dict(position_offset=int(position_offset), interleaved=bool(interleaved),
                eps=None if eps is None else float(eps))
    return _QkNormRope.apply(q, k, q_weight, k_weight, inv_freq, positions, opts)


def _cache(p, k_cache, v_cache, Hk, d, device):
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must both be [n_pages, Hk, page_size, d]")
    pages, _, page, _ = k_cache.shape
    p.k_cache_stride[:] = _heads("k_cache", k_cache, (pages, Hk, page, d))
    p.v_cache_stride[:] = _heads("v_cache", v_cache, (pages, Hk, page, d))
    _same_device(device, k_cache=k_cache, v_cache=v_cache)
    p.n_pages, p.page_size = pages, page


def _plan_append(k, v, k_cache, v_cache, block_table, starts, counts, positions, inv_freq, interleaved, eps, k_weight,
                 q, q_weight, q_out):
    if k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, Hk, N, d = k.shape
    device = k.device
    p = _lib.AttnRopeParams()
    p.B, p.N, p.Hk, p.d = B, N, Hk, d
    p.k_stride[:] = _heads("k", k)
    p.v_stride[:] = _heads("v", v, k.shape)
    _same_device(device, v=v, q=q, q_out=q_out)
    _cache(p, k_cache, v_cache, Hk, d, device)
    _int32("block_table", block_table, device, (B, None))
    p.table_width, p.table_stride = block_table.shape[1], block_table.stride(0)
    _int32("starts", starts, device, (B,))
    if counts is not None:
        _int32("counts", counts, device, (B,))
    if q is not None:
        if q.dim() != 4:
            raise ValueError("expected [B, H, N, d] tensors")
        p.Hq = q.shape[1]
        p.q_stride[:] = _heads("q", q, (B, p.Hq, N, d))
    elif q_weight is not None or q_out is not None:
        raise ValueError("q_weight and q_out need q")
    _set_rope(p, B, N, d, device, q_weight, k_weight, inv_freq, positions, interleaved, eps)
    if q_out is not None:
        p.q_out_stride[:] = _heads("q_out", q_out, q.shape)
    return bytes(p)


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_table: torch.Tensor, starts: torch.Tensor, *, counts: torch.Tensor | None = None,
              position_offset: int = 0, positions: torch.Tensor | None = None,
              inv_freq: torch.Tensor | None = None, interleaved: bool = False, eps: float | None = None,
              k_weight: torch.Tensor | None = None, q: torch.Tensor | None = None,
              q_weight: torch.Tensor | None = None, q_out: torch.Tensor | None = None, stream=None):
    """Appends N new tokens of every sequence to a paged cache, in place.

    k, v [B, Hk, N, d]; k_cache, v_cache [n_pages, Hk, page_size, d] (page_size a power
    of two from 16); block_table [B, width] pages of each sequence; starts [B] tokens
    that each holds already. Token n goes to slot starts[b] + n. Keys are normed (eps
    given; k_weight) and rotated (inv_freq) on the way as qk_norm_rope_fwd does, at
    `positions`, else at position_offset + starts[b] + n (position_offset: the length of
    a shared prefix). With `q` [B, Hq, N, d] the same tokens' queries are normed and
    rotated in the same launch and returned (in q_out if given); else returns None.

    counts [B]: real tokens of each sequence; those behind leave the cache as it was, as
    do negative starts, slots behind the table's end and entries that are not a page of
    the cache. The pages that a call writes must not be shared between sequences.
    No gradient goes through it.
    """
    interleaved, eps = bool(interleaved), None if eps is None else float(eps)
    key = ("append", _sig(k), _sig(v), _sig(k_cache), _sig(v_cache), _sig(block_table), _sig(starts), _sig(counts),
           _sig(positions), _sig(inv_freq), interleaved, eps, _sig(k_weight), _sig(q), _sig(q_weight), _sig(q_out))
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_append(k, v, k_cache, v_cache, block_table, starts, counts, positions, inv_freq,
                                           interleaved, eps, k_weight, q, q_weight, q_out))
    device = k.device
    p = _lib.AttnRopeParams.from_buffer_copy(plan)
    p.q, p.k, p.v, p.k_cache, p.v_cache = _ptr(q), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    p.block_table, p.starts, p.counts = block_table.data_ptr(), starts.data_ptr(), _ptr(counts)
    p.q_weight, p.k_weight = _ptr(q_weight), _ptr(k_weight)
    p.inv_freq, p.positions = _ptr(inv_freq), _ptr(positions)
    p.pos_offset = _fits("position_offset", int(position_offset), 64)

    def run(handle):
        qo = q_out
        if q is not None:
            if qo is None:
                qo = torch.empty(q.shape, dtype=torch.bfloat16, device=device)
            p.q_out = qo.data_ptr()
        p.stream = handle
        code = _lib.load().attn_kv_append(ctypes.byref(p))
        if code:
            _lib.check(code, "kv_append")
        _wrote((k_cache, v_cache) if q_out is None else (k_cache, v_cache, q_out))
        return qo

    return _on(device, stream, (k, v, k_cache, v_cache, block_table, starts, counts, positions, inv_freq, k_weight, q,
                                q_weight, q_out), run)


_PAGED_MASKS = {"none": _lib.ATTN_MASK_NONE, "causal_br": _lib.ATTN_MASK_CAUSAL_BR}


def _plan_paged(q, k_cache, v_cache, block_table, kv_lens, q_lens, prefix_table, prefix_len, scale, mask, out, lse,
                num_ctas):
    """(the parameter block, bytes of workspace)"""
    if mask not in _PAGED_MASKS:
        raise ValueError(f"mask must be 'none' or 'causal_br', not {mask!r}")
    _fits("prefix_len", prefix_len)
    _fits("num_ctas", num_ctas)
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, Hq, Nq, d = q.shape
    device = q.device
    p = _lib.AttnPagedParams()
    p.q_stride[:] = _heads("q", q)
    if k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must both be [n_pages, Hk, page_size, d]")
    p.B, p.Hq, p.Hk, p.Nq, p.d = B, Hq, k_cache.shape[1], Nq, d
    _cache(p, k_cache, v_cache, p.Hk, d, device)
    _int32("block_table", block_table, device, (B, None))
    p.table_width, p.table_stride = block_table.shape[1], block_table.stride(0)
    _int32("kv_lens", kv_lens, device, (B,))
    if q_lens is not None:
        _int32("q_lens", q_lens, device, (B,))
    p.prefix_len = prefix_len
    if prefix_table is not None:
        _int32("prefix_table", prefix_table, device, (None,))
        p.prefix_pages = prefix_table.shape[0]
    p.scale = float(1.0 / math.sqrt(d) if scale is None else scale)
    p.mask_kind = _PAGED_MASKS[mask]
    p.num_ctas = num_ctas
    _same_device(device, out=out, lse=lse)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != (B, Hq, Nq)):
        raise ValueError("lse must be a contiguous float32 [B, Hq, Nq] tensor")
    if out is not None:
        p.o_stride[:] = _heads("out", out, q.shape)
    with torch.cuda.device(device):
        n = _lib.load().attn_paged_workspace_bytes(ctypes.byref(p))
    if n < 0:
        _lib.check(int(-n), "attn_paged")
    return bytes(p), int(n)


def attn_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
               kv_lens: torch.Tensor, *, q_lens: torch.Tensor | None = None,
               prefix_table: torch.Tensor | None = None, prefix_len: int = 0, scale: float | None = None,
               mask: str = "causal_br", out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               return_lse: bool = True, num_ctas: int = 0, timeout_ns: int = 0, inject: int = 0, stream=None):
    """Attention of a batch of sequences over a paged cache, with a shared prefix.

    q [B, Hq, Nq, d]; k_cache, v_cache [n_pages, Hk, page_size, d], Hq a multiple of Hk
    (query head h reads key head h // (Hq // Hk)). The keys of sequence b are the first
    prefix_len tokens of the pages in prefix_table (one table for the whole batch; its
    keys are read once per 256 query rows of a key head, of all sequences together, where
    that pays, else by each sequence), then kv_lens[b] tokens of the pages in block_table[b].
    Its queries are the last q_lens[b] of these tokens (None: Nq); rows behind q_lens[b]
    are padding. mask 'causal_br': row i sees keys up to i + T - q_lens[b], T = prefix_len
    + kv_lens[b]; 'none': every real row sees all T. A row that sees no key (or only
    scores of -inf) gives 0 and an LSE of -inf, one with a score that is NaN or +inf NaN
    for both. Values (v_cache) of keys that only some rows of a sequence see must be
    finite. Lengths and tables are read when the kernels run.

    Returns (o, lse) or o; no gradient goes through it. Raises for what the host can
    check; a bad table entry reads as zeros, a length beyond the table's end is cut.
    """
    prefix_len, num_ctas = int(prefix_len), int(num_ctas)  # (what a key holds is a value, never a tensor)
    timeout_ns, inject = _fits("timeout_ns", int(timeout_ns), 64), _fits("inject", int(inject))
    if timeout_ns < 0:
        raise ValueError("timeout_ns must be >= 0")
    scale = None if scale is None else float(scale)
    key = ("paged", _sig(q), _sig(k_cache), _sig(v_cache), _sig(block_table), _sig(kv_lens), _sig(q_lens),
           _sig(prefix_table), prefix_len, scale, mask, _sig(out), _sig(lse), num_ctas)
    plan = _plans.get(key)
    if plan is None:
        plan = _remember(key, _plan_paged(q, k_cache, v_cache, block_table, kv_lens, q_lens, prefix_table, prefix_len,
                                          scale, mask, out, lse, num_ctas))
    device = q.device
    p = _lib.AttnPagedParams.from_buffer_copy(plan[0])
    p.q, p.k_cache, p.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    p.block_table, p.kv_lens, p.q_lens = block_table.data_ptr(), kv_lens.data_ptr(), _ptr(q_lens)
    p.prefix_table, p.timeout_ns, p.inject = _ptr(prefix_table), timeout_ns, inject

    def run(handle):
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=device) if out is None else out
        p.o = o.data_ptr()
        z = lse
        if z is None and return_lse:
            z = torch.empty(q.shape[:3], dtype=torch.float32, device=device)
        if z is not None:
            p.lse = z.data_ptr()
        ws = torch.empty(plan[1], dtype=torch.uint8, device=device)
        p.workspace, p.workspace_bytes = ws.data_ptr(), plan[1]
        p.stream = handle
        code = _lib.load().attn_paged(ctypes.byref(p))
        if code:
            _lib.check(code, "attn_paged")
        if out is not None or lse is not None:
            _wrote([t for t in (out, lse) if t is not None])
        return (o, z) if return_lse else o

    return _on(device, stream, (q, k_cache, v_cache, block_table, kv_lens, q_lens, prefix_table, out, lse), run)
