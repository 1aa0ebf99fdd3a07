"""GPU: the per-head norm with rotation, its gradient and the cache append
against their definitions in 64 bits (bounds in cache_oracle)."""
import math

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


def weight(seed, d, dtype):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)


# B, Hq, Hk, N, d, rot, interleaved, eps, first position
FWD = [
    (1, 1, 1, 1, 32, 32, False, 1e-6, 0),
    (1, 1, 1, 1, 128, 128, True, 1e-6, 5),
    (2, 5, 5, 77, 64, 32, True, 1e-6, 1000),
    (2, 5, 1, 77, 64, 32, False, 1e-5, 1000),
    (3, 8, 2, 33, 128, 128, False, 1e-6, 131071),
    (1, 7, 1, 130, 128, 64, False, None, 10 ** 6),
    (2, 3, 3, 19, 32, 16, True, None, 3),
    (1, 2, 2, 65, 64, 0, False, 1e-6, 0),
    (5, 4, 0, 9, 128, 128, False, 1e-6, 2 ** 31),
    (1, 40, 8, 300, 128, 128, False, 1e-6, 17),
]


@pytest.mark.parametrize("case", FWD, ids=str)
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32, None], ids=["wbf16", "wfp32", "now"])
def test_forward(E, case, wtype):
    B, Hq, Hk, N, d, rot, il, eps, first = case
    q, k = rnd(1, B, Hq, N, d, scale=3.0), rnd(2, B, max(Hk, 1), N, d)
    wq = wk = None
    if wtype is not None and eps is not None:
        wq, wk = weight(3, d, wtype), weight(4, d, wtype)
    freqs = E.rope_freqs(rot, device="cpu") if rot else None
    pos = first + torch.arange(N)[None, :].expand(B, N) * 3 + torch.arange(B)[:, None]
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    qo, ko = E.qk_norm_rope_fwd(q.cuda(), k.cuda() if Hk else None, cu(wq), cu(wk) if Hk else None, inv_freq=cu(freqs),
                                positions=pos.cuda(), interleaved=il, eps=eps)
    O.check("q", qo, *O.norm_rope(q, wq, pos, freqs, il, eps))
    if Hk:
        O.check("k", ko, *O.norm_rope(k, wk, pos, freqs, il, eps))


def test_default_positions_strides_and_in_place(E):
    """Views of a fused projection, int32 shared positions, outputs into given heads-last
    tensors and over the inputs themselves."""
    B, Hq, Hk, N, d = 2, 6, 2, 45, 64
    x = rnd(5, B, N, Hq + 2 * Hk, d)
    freqs = E.rope_freqs(d, base=500000.0)
    xc = x.cuda()
    qc, kc = xc[:, :, :Hq].transpose(1, 2), xc[:, :, Hq:Hq + Hk].transpose(1, 2)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    pos = (torch.arange(N) + 7)[None].expand(B, N)
    want_q, want_k = (O.norm_rope(t, None, pos, freqs.cpu(), False, 1e-6) for t in (q, k))
    qo, ko = E.qk_norm_rope_fwd(qc, kc, inv_freq=freqs, position_offset=7)
    O.check("q", qo, *want_q)
    O.check("k", ko, *want_k)
    out = torch.full((B, N, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    qo2, _ = E.qk_norm_rope_fwd(qc, kc, inv_freq=freqs, positions=pos[0].to(torch.int32).cuda(), q_out=out)
    assert qo2.data_ptr() == out.data_ptr() and torch.equal(out, qo)
    E.qk_norm_rope_fwd(qc, kc, inv_freq=freqs, position_offset=7, q_out=qc, k_out=kc)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)
    assert torch.equal(xc[:, :, Hq + Hk:].cpu(), x[:, :, Hq + Hk:]), "the values beside them stay"


def test_expanded_input_and_zero_row(E):
    """One head expanded to five, and a row of zeros: eps keeps it finite."""
    q = rnd(6, 1, 1, 4, 32)
    q[0, 0, 2] = 0
    qo, _ = E.qk_norm_rope_fwd(q.cuda().expand(1, 5, 4, 32), None, inv_freq=E.rope_freqs(32))
    want = O.norm_rope(q.expand(1, 5, 4, 32), None, torch.arange(4)[None], E.rope_freqs(32, device="cpu"), False, 1e-6)
    O.check("q", qo, *want)
    assert float(qo[0, :, 2].abs().max()) == 0.0


def test_negative_positions_and_fast_frequencies(E):
    """The fixed-point angle wraps for negative positions and drops whole turns of a
    frequency above one turn a position."""
    freqs = torch.tensor([1.0, -0.3, 7.5, 1e-9, 100.25, 0.0, 2 * math.pi, 1e-300], dtype=torch.float64)
    q = rnd(7, 1, 2, 6, 32)
    pos = torch.tensor([[-5, -1, 0, 1, 123456, -99999]])
    qo, _ = E.qk_norm_rope_fwd(q.cuda(), None, inv_freq=freqs.cuda(), positions=pos.cuda())
    O.check("q", qo, *O.norm_rope(q, None, pos, freqs, False, 1e-6))


@pytest.mark.parametrize("case", [c for c in FWD if c[2] > 0], ids=str)
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32], ids=["wbf16", "wfp32"])
def test_backward(E, case, wtype):
    B, Hq, Hk, N, d, rot, il, eps, first = case
    q, k = rnd(11, B, Hq, N, d, scale=2.0), rnd(12, B, Hk, N, d)
    gq, gk = rnd(13, B, Hq, N, d), rnd(14, B, Hk, N, d)
    wq, wk = (weight(15, d, wtype), weight(16, d, wtype)) if eps is not None else (None, None)
    freqs = E.rope_freqs(rot, device="cpu") if rot else None
    pos = first + torch.arange(N)[None, :].expand(B, N)
    leaves = [t.cuda().requires_grad_() for t in (q, k, wq, wk) if t is not None]
    w = leaves[2:] if len(leaves) == 4 else [None, None]
    qo, ko = E.qk_norm_rope(leaves[0], leaves[1], *w, inv_freq=None if freqs is None else freqs.cuda(),
                            position_offset=first, interleaved=il, eps=eps)
    grads = torch.autograd.grad((qo, ko), leaves, (gq.cuda(), gk.cuda()))
    for i, (x, ww, g) in enumerate(((q, wq, gq), (k, wk, gk))):
        dx, bx, dw, bw = O.norm_rope_back(x, ww, g, pos, freqs, il, eps)
        O.check("dx", grads[i], dx, bx)
        if ww is not None:
            assert grads[2 + i].dtype == wtype
            O.check("dw", grads[2 + i], dw, bw)


def test_backward_one_output_and_expanded_gradient(E):
    """A loss that reaches only one output, with an expanded gradient; and the same bits
    twice (no atomics)."""
    q, k = rnd(31, 2, 4, 50, 64), rnd(32, 2, 2, 50, 64)
    w = weight(33, 64, torch.float32)
    pos, freqs = torch.arange(50)[None].expand(2, 50), E.rope_freqs(64, device="cpu")
    got = []
    for _ in range(2):
        leaves = [t.cuda().requires_grad_() for t in (q, k, w, w)]
        qo, ko = E.qk_norm_rope(*leaves, inv_freq=freqs.cuda())
        ko.sum().backward()
        assert leaves[0].grad is None and leaves[2].grad is None
        got.append((leaves[1].grad, leaves[3].grad))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    dx, bx, dw, bw = O.norm_rope_back(k, w, torch.ones_like(k), pos, freqs, False, 1e-6)
    O.check("dk", got[0][0], dx, bx)
    O.check("dwk", got[0][1], dw, bw)


# B, Hq, Hk, N, d, page, interleaved, eps, ragged
APPEND = [
    (1, 0, 1, 1, 32, 16, False, None, False),
    (3, 4, 2, 1, 128, 16, False, 1e-6, False),
    (4, 6, 2, 37, 64, 32, True, None, True),
    (2, 5, 5, 130, 128, 64, False, 1e-6, True),
    (3, 7, 1, 9, 32, 256, True, 1e-6, False),
]


def pages_for(lens, page, extra_pages, seed):
    g = torch.Generator().manual_seed(seed)
    need = [max(1, -(-n // page)) for n in lens]
    order = torch.randperm(sum(need) + extra_pages, generator=g).tolist()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table, order[at:], len(order)


@pytest.mark.parametrize("nhd", [False, True], ids=["hnd", "nhd"])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(E, case, nhd):
    B, Hq, Hk, N, d, page, il, eps, ragged = case
    starts = [(13 * b * b + 5 * b) % 70 for b in range(B)]
    table, _, n_pages = pages_for([s + N for s in starts], page, 2, 41)
    x = rnd(42, B, N, Hq + 2 * Hk, d)
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    kc, vc = rnd(43, n_pages, Hk, page, d), rnd(44, n_pages, Hk, page, d)
    counts = torch.tensor([max(0, N - 4 * b - 1) for b in range(B)], dtype=torch.int32) if ragged else None
    wq, wk = (weight(45, d, torch.float32), weight(46, d, torch.bfloat16)) if eps is not None else (None, None)
    freqs = E.rope_freqs(d, device="cpu")
    offset = 1021
    xc = x.cuda()
    kcc, vcc = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if nhd else t.cuda() for t in (kc, vc))
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    qo = E.kv_append(xc[:, :, Hq:Hq + Hk].transpose(1, 2), xc[:, :, Hq + Hk:].transpose(1, 2), kcc, vcc, table.cuda(),
                     torch.tensor(starts, dtype=torch.int32).cuda(), counts=cu(counts), position_offset=offset,
                     inv_freq=freqs.cuda(), interleaved=il, eps=eps, k_weight=cu(wk),
                     q=xc[:, :, :Hq].transpose(1, 2) if Hq else None, q_weight=cu(wq) if Hq else None)
    pos = offset + torch.tensor(starts)[:, None] + torch.arange(N)
    want_k, kb, want_v = O.append(k, v, kc, vc, table, starts, counts, pos, freqs, il, eps, wk)
    O.check("k_cache", kcc, want_k, kb)
    O.check("v_cache", vcc, want_v, torch.zeros_like(want_v))
    if Hq:
        O.check("q", qo, *O.norm_rope(q, wq, pos, freqs, il, eps))
    else:
        assert qo is None


def test_append_leaves_the_rest(E):
    """Negative starts, entries that are no page, slots behind the table: nothing is
    written; NaN in tokens behind the count stays out."""
    B, Hk, N, d, page = 5, 2, 20, 64, 16
    table = torch.tensor([[0, 1], [2, 99], [3, -1], [4, 5], [6, 7]], dtype=torch.int32)
    starts = torch.tensor([5, 10, 12, -3, 30], dtype=torch.int32)
    counts = torch.tensor([20, 20, 20, 20, 7], dtype=torch.int32)
    k, v = rnd(51, B, Hk, N, d), rnd(52, B, Hk, N, d)
    k[4, :, 7:] = float("nan")
    v[4, :, 7:] = float("nan")
    kc, vc = rnd(53, 8, Hk, page, d), rnd(54, 8, Hk, page, d)
    kcc, vcc = kc.cuda(), vc.cuda()
    E.kv_append(k.cuda(), v.cuda(), kcc, vcc, table.cuda(), starts.cuda(), counts=counts.cuda())
    want_k, kb, want_v = O.append(k, v, kc, vc, table, starts, counts, torch.zeros(B, N), None, False, None, None)
    O.check("k_cache", kcc, want_k, torch.zeros_like(kb))
    O.check("v_cache", vcc, want_v, torch.zeros_like(want_v))


def test_queries_alone_and_no_rotation(E):
    """k None through autograd; norm without rotation; rotation without norm (its own
    gradient is the inverse rotation)."""
    q, g = rnd(81, 2, 3, 11, 64), rnd(82, 2, 3, 11, 64)
    pos, freqs = torch.arange(11)[None].expand(2, 11), E.rope_freqs(64, device="cpu")
    for f, eps in ((None, 1e-6), (freqs, None), (freqs, 1e-6)):
        x = q.cuda().requires_grad_()
        y, none = E.qk_norm_rope(x, None, inv_freq=None if f is None else f.cuda(), eps=eps)
        assert none is None
        (dx,) = torch.autograd.grad(y, x, g.cuda())
        O.check("y", y, *O.norm_rope(q, None, pos, f, False, eps))
        O.check("dx", dx, *O.norm_rope_back(q, None, g, pos, f, False, eps)[:2])


def test_two_streams_at_once(E):
    """Two gradients at once have their own scratch."""
    q, g, w = rnd(83, 2, 8, 600, 128).cuda(), rnd(84, 2, 8, 600, 128).cuda(), weight(85, 128, torch.float32).cuda()
    f = E.rope_freqs(128)
    want = E.qk_norm_rope_bwd(q, None, g, None, w, inv_freq=f)
    other = E.qk_norm_rope_bwd(g, None, q, None, w, inv_freq=f)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a = E.qk_norm_rope_bwd(q, None, g, None, w, inv_freq=f, stream=s1)
        b = E.qk_norm_rope_bwd(g, None, q, None, w, inv_freq=f, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a[0], want[0]) and torch.equal(a[2], want[2])
        assert torch.equal(b[0], other[0]) and torch.equal(b[2], other[2])


def test_refusals(E):
    q, k = rnd(86, 1, 4, 5, 64).cuda(), rnd(87, 1, 2, 5, 64).cuda()
    w, f = weight(88, 64, torch.float32).cuda(), E.rope_freqs(64)
    for args, kw in (((q.float(), k), {}), ((q[0], k), {}), ((q, k[:, :, :4]), {}), ((q, k, w[:32]), {}),
                     ((q, k, w.double()), {}), ((q, k, w), dict(eps=None)), ((q, k), dict(inv_freq=f.float())),
                     ((q, k), dict(inv_freq=f.cpu())), ((q, k), dict(inv_freq=f, positions=torch.zeros(4, device="cuda").long())),
                     ((q, k), dict(inv_freq=f, positions=torch.zeros(5, device="cuda"))), ((q, k), dict(k_out=q)),
                     ((q.transpose(2, 3), k), {}), ((q, None, None, w), {})):
        with pytest.raises((TypeError, ValueError)):
            E.qk_norm_rope_fwd(*args, **kw)
    for kw in (dict(inv_freq=E.rope_freqs(128)), dict(inv_freq=f[:4].contiguous()), dict(eps=float("nan"))):
        with pytest.raises(E.AttnError):
            E.qk_norm_rope_fwd(q, k, **kw)
    with pytest.raises(E.AttnError):  # a view that starts off a 16-byte boundary
        E.qk_norm_rope_fwd(torch.zeros(1, 1, 5, 72, dtype=torch.bfloat16, device="cuda")[..., 4:68], None)
    x = q.clone().requires_grad_()
    y, _ = E.qk_norm_rope(x, k, inv_freq=f)
    (dx,) = torch.autograd.grad(y, x, torch.ones_like(y, requires_grad=True), create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_side_stream_and_graph(E):
    """On a given stream, and captured: the replay follows new starts."""
    B, Hk, N, d, page = 2, 2, 3, 64, 16
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    k, v = rnd(61, B, Hk, N, d), rnd(62, B, Hk, N, d)
    kc = torch.zeros(4, Hk, page, d, dtype=torch.bfloat16)
    freqs = E.rope_freqs(d)
    s = torch.cuda.Stream()
    kd, vd, td = k.cuda(), v.cuda(), table.cuda()
    starts = torch.tensor([0, 9], dtype=torch.int32).cuda()
    kcc, vcc = kc.cuda(), kc.cuda()
    s.wait_stream(torch.cuda.current_stream())
    E.kv_append(kd, vd, kcc, vcc, td, starts, inv_freq=freqs, stream=s)
    torch.cuda.current_stream().wait_stream(s)

    def want(st):
        pos = torch.tensor(st)[:, None] + torch.arange(N)
        return O.append(k, v, kc, kc, table, st, None, pos, freqs.cpu(), False, None, None)

    wk, kb, wv = want([0, 9])
    O.check("k", kcc, wk, kb)
    O.check("v", vcc, wv, torch.zeros_like(wv))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.kv_append(kd, vd, kcc, vcc, td, starts, inv_freq=freqs)
    for st in ([14, 0], [3, 27]):
        kcc.zero_()
        vcc.zero_()
        starts.copy_(torch.tensor(st, dtype=torch.int32))
        g.replay()
        wk, kb, wv = want(st)
        O.check("k", kcc, wk, kb)
        O.check("v", vcc, wv, torch.zeros_like(wv))


def test_backward_captured(E):
    """A whole training step of the op captured and replayed with new inputs (no eager
    graph of the same leaves alive)."""
    q, k, g = rnd(71, 1, 3, 40, 64), rnd(72, 1, 1, 40, 64), rnd(73, 1, 3, 40, 64)
    w = weight(74, 64, torch.float32)
    freqs = E.rope_freqs(64)
    qs, ks, ws = (t.cuda().requires_grad_() for t in (q, k, w))
    gd = g.cuda()

    def step():
        qo, ko = E.qk_norm_rope(qs, ks, ws, None, inv_freq=freqs)
        return torch.autograd.grad((qo, ko), (qs, ks, ws), (gd, gd[:, :1]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    q2 = rnd(75, 1, 3, 40, 64)
    with torch.no_grad():
        qs.copy_(q2)
    graph.replay()
    pos = torch.arange(40)[None]
    dx, bx, dw, bw = O.norm_rope_back(q2, w, g, pos, freqs.cpu(), False, 1e-6)
    O.check("dq", out[0], dx, bx)
    O.check("dw", out[2], dw, bw)
