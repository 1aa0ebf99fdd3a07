"""GPU: the norm with rotation and the cache append in forms that their callers meet less
often, against the definitions in 64 bits (bounds in cache_oracle)."""
import pytest
import torch

from tests import cache_oracle as O
from tests.test_gpu_rope import E, rnd, weight  # noqa: F401  (E: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [1, 4, 8])
def test_gradient_off_a_16_byte_boundary(E, off):  # noqa: F811
    """Incoming gradients that are contiguous slices of a flat buffer, anywhere in it."""
    q, k, gq, gk = (rnd(100 + i, 2, h, 7, 64) for i, h in enumerate((4, 2, 4, 2)))
    pos, freqs = torch.arange(7)[None].expand(2, 7), E.rope_freqs(64)
    flat = torch.cat([torch.zeros(off, dtype=torch.bfloat16), gq.flatten(), gk.flatten()]).cuda()
    dq = flat[off:off + gq.numel()].view(gq.shape)
    dk = flat[off + gq.numel():].view(gk.shape)
    assert dq.is_contiguous() and (dq.data_ptr() % 16 != 0) == (off % 8 != 0)
    x, y = q.cuda().requires_grad_(), k.cuda().requires_grad_()
    got = torch.autograd.grad(E.qk_norm_rope(x, y, inv_freq=freqs), (x, y), (dq, dk))
    for have, a, g in zip(got, (q, k), (gq, gk)):
        O.check("dx", have, *O.norm_rope_back(a, None, g, pos, freqs.cpu(), False, 1e-6)[:2])


def test_offsets_that_do_not_fit(E):  # noqa: F811
    """position_offset is a signed 64-bit number: its ends are taken, beyond them it is refused."""
    q = rnd(110, 1, 2, 1, 64)
    f = E.rope_freqs(64)
    c, table, one = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16, device="cuda"), *(
        torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 1), (1,)))
    for bad in (2 ** 63, -2 ** 63 - 1, 2 ** 64 + 5):
        with pytest.raises(ValueError, match="position_offset"):
            E.qk_norm_rope_fwd(q.cuda(), None, inv_freq=f, position_offset=bad)
        with pytest.raises(ValueError, match="position_offset"):
            E.qk_norm_rope_bwd(q.cuda(), None, q.cuda(), None, inv_freq=f, position_offset=bad)
        with pytest.raises(ValueError, match="position_offset"):
            E.kv_append(q.cuda(), q.cuda(), c, c.clone(), table, one, inv_freq=f, position_offset=bad)
    # (the 64-bit fixed point is exact to position * 2^-64 of a turn: at 2^40 to 2^-21.3 radians)
    few = torch.tensor([1.0, 0.5, -0.75, 2.0 ** -9, 3 * 2.0 ** -30, 1.25, 2.0 ** -40, 0.375], dtype=torch.float64)
    for far in (2 ** 40 + 3, -2 ** 40 - 1):
        y, _ = E.qk_norm_rope_fwd(q.cuda(), None, inv_freq=few.cuda(), position_offset=far)
        O.check("y", y, *O.norm_rope(q, None, torch.tensor([[far]]), few, False, 1e-6))
    for end in (2 ** 63 - 1, -2 ** 63):
        y, _ = E.qk_norm_rope_fwd(q.cuda(), None, inv_freq=few.cuda(), position_offset=end)
        assert bool(torch.isfinite(y).all())


def test_written_tensors_are_known_to_autograd(E):  # noqa: F811
    """A graph that saved a tensor which a later call writes refuses its backward pass."""
    q, k = rnd(120, 1, 2, 20, 64).cuda(), rnd(121, 1, 2, 20, 64).cuda()
    f = E.rope_freqs(64)
    table, one = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = one + 20
    cache = lambda: torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def saved(t):  # a graph that keeps t
        w = torch.ones((), device="cuda", dtype=t.dtype, requires_grad=True)
        return (w * t).sum()

    def refused(loss):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()

    x = q.clone().requires_grad_()
    y, _ = E.qk_norm_rope(x, None, inv_freq=f)
    with torch.no_grad():
        E.qk_norm_rope_fwd(x, k, inv_freq=f, q_out=x)
    refused(y.float().sum())
    k2 = k.clone()
    loss = saved(k2)
    E.qk_norm_rope_fwd(q, k2, inv_freq=f, k_out=k2)
    refused(loss)
    kc, vc, qo = cache(), cache(), torch.empty_like(q)
    losses = [saved(t) for t in (kc, vc, qo)]
    E.kv_append(k, k, kc, vc, table, one, q=q, q_out=qo)
    for loss in losses:
        refused(loss)
    o, z = torch.empty_like(q), torch.empty(1, 2, 20, device="cuda")
    losses = [saved(t) for t in (o, z)]
    kept = saved(kc)  # read, not written
    E.attn_paged(q, kc, vc, table, lens, out=o, lse=z)
    for loss in losses:
        refused(loss)
    kept.backward()
    with torch.inference_mode():
        E.kv_append(k, k, cache(), cache(), table, one, q=q, q_out=torch.empty_like(q))


@pytest.mark.parametrize("needs", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (1, 1, 0, 1), (1, 0, 0, 1),
                                   (0, 0, 1, 1), (1, 1, 1, 1)], ids=str)
def test_only_the_gradients_that_are_asked_for(E, needs, monkeypatch):  # noqa: F811
    """Sides and weights that need no gradient are left out of the call; what is asked for
    does not depend on the rest."""
    from exact_attention_69_gb300 import cache
    q, k, gq, gk = (rnd(130 + i, 2, h, 19, 64) for i, h in enumerate((4, 2, 4, 2)))
    wq, wk = weight(134, 64, torch.float32), weight(135, 64, torch.bfloat16)
    pos, freqs = torch.arange(19)[None].expand(2, 19), E.rope_freqs(64)
    calls, real = [], cache.qk_norm_rope_bwd

    def spy(*a, **kw):
        out = real(*a, **kw)
        calls.append((a, out))
        return out

    monkeypatch.setattr(cache, "qk_norm_rope_bwd", spy)
    ts = [t.cuda().requires_grad_(bool(n)) for t, n in zip((q, k, wq, wk), needs)]
    got = torch.autograd.grad(E.qk_norm_rope(*ts, inv_freq=freqs), [t for t in ts if t.requires_grad], (gq.cuda(), gk.cuda()))
    (args, out), = calls
    sides = (needs[0] or needs[2]) + (needs[1] or needs[3])
    assert (args[1] is not None) == (sides == 2)
    assert sum(t is not None for t in out[2:]) == needs[2] + needs[3]
    bq, bk = (O.norm_rope_back(x, w, g, pos, freqs.cpu(), False, 1e-6) for x, w, g in ((q, wq, gq), (k, wk, gk)))
    want = [bq[:2], bk[:2], bq[2:], bk[2:]]
    for have, (ref, bound) in zip(got, [w for w, n in zip(want, needs) if n]):
        O.check("gradient", have, ref, bound)


@pytest.mark.parametrize("form", ["int32 [N]", "int64 [B, N]", "int32 [N, B] transposed", "int64 [N] every third"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_gradient_with_positions(E, form, interleaved):  # noqa: F811
    """The gradient turns back by the positions that the forward was given, not by an offset."""
    B, N = 3, 21
    q, k, gq, gk = (rnd(140 + i, B, h, N, 64) for i, h in enumerate((4, 2, 4, 2)))
    w = weight(144, 64, torch.bfloat16)
    g = torch.Generator().manual_seed(145)
    if form == "int32 [N]":
        pos = torch.randint(-500, 10 ** 6, (N,), generator=g).to(torch.int32)
        given = pos.cuda()
    elif form == "int64 [B, N]":
        pos = torch.randint(-500, 10 ** 6, (B, N), generator=g)
        given = pos.cuda()
    elif form == "int32 [N, B] transposed":
        pos = torch.randint(0, 10 ** 6, (N, B), generator=g).to(torch.int32)
        given, pos = pos.cuda().t(), pos.t()
    else:
        pos = torch.randint(0, 10 ** 6, (3 * N,), generator=g)
        given, pos = pos.cuda()[::3], pos[::3]
    full = pos.expand(B, N) if pos.dim() == 1 else pos
    freqs = E.rope_freqs(32)
    x, y, ww = q.cuda().requires_grad_(), k.cuda().requires_grad_(), w.cuda().requires_grad_()
    out = E.qk_norm_rope(x, y, ww, None, inv_freq=freqs, positions=given, position_offset=99, interleaved=interleaved)
    O.check("q", out[0], *O.norm_rope(q, w, full, freqs.cpu(), interleaved, 1e-6))
    dq, dk, dw = torch.autograd.grad(out, (x, y, ww), (gq.cuda(), gk.cuda()))
    rq, bq, rw, bw = O.norm_rope_back(q, w, gq, full, freqs.cpu(), interleaved, 1e-6)
    O.check("dq", dq, rq, bq)
    O.check("dw", dw, rw, bw)
    O.check("dk", dk, *O.norm_rope_back(k, None, gk, full, freqs.cpu(), interleaved, 1e-6)[:2])


@pytest.mark.parametrize("eps", [None, 1e-6], ids=["plain", "norm"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("d,rot", [(32, 16), (64, 32), (64, 48), (128, 64), (128, 16)])
def test_append_partly_rotated(E, d, rot, interleaved, eps):  # noqa: F811
    """Fewer rotated channels than a head has, into the cache and beside it."""
    B, Hq, Hk, N, page = 2, 3, 1, 19, 16
    starts = [5, 30]
    table = torch.tensor([[4, 0, 9], [2, 7, 1], ], dtype=torch.int32)
    table = torch.cat([table, torch.tensor([[3], [5]], dtype=torch.int32)], 1)
    q, k, v = rnd(150, B, Hq, N, d), rnd(151, B, Hk, N, d), rnd(152, B, Hk, N, d)
    kc, vc = rnd(153, 10, Hk, page, d), rnd(154, 10, Hk, page, d)
    wk = weight(155, d, torch.bfloat16) if eps is not None else None
    freqs = E.rope_freqs(rot)
    kcc, vcc = kc.cuda(), vc.cuda()
    qo = E.kv_append(k.cuda(), v.cuda(), kcc, vcc, table.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
                     position_offset=77, inv_freq=freqs, interleaved=interleaved, eps=eps,
                     k_weight=None if wk is None else wk.cuda(), q=q.cuda())
    pos = 77 + torch.tensor(starts)[:, None] + torch.arange(N)
    want_k, kb, want_v = O.append(k, v, kc, vc, table, starts, None, pos, freqs.cpu(), interleaved, eps, wk)
    O.check("k_cache", kcc, want_k, kb)
    O.check("v_cache", vcc, want_v, torch.zeros_like(want_v))
    O.check("q", qo, *O.norm_rope(q, None, pos, freqs.cpu(), interleaved, eps))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["int32", "int64"])
@pytest.mark.parametrize("shared", [False, True], ids=["own", "shared"])
def test_append_with_positions_and_outputs(E, dtype, shared):  # noqa: F811
    """Positions that are not the slots, [B, N] and [N]; queries into a heads-last tensor, and
    over themselves inside a fused projection."""
    B, Hq, Hk, N, d, page = 3, 4, 2, 11, 64, 16
    starts = [0, 20, 9]
    table = torch.tensor([[0, 1], [6, 3], [4, 5]], dtype=torch.int32)
    x = rnd(160, B, N, Hq + 2 * Hk, d)
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    kc, vc = rnd(161, 7, Hk, page, d), rnd(162, 7, Hk, page, d)
    g = torch.Generator().manual_seed(163)
    pos = torch.randint(0, 2 ** 31 - 1, (N,) if shared else (B, N), generator=g).to(dtype)
    full = pos.expand(B, N)
    freqs = E.rope_freqs(d)
    want_k, kb, want_v = O.append(k, v, kc, vc, table, starts, None, full, freqs.cpu(), False, 1e-6, None)
    want_q = O.norm_rope(q, None, full, freqs.cpu(), False, 1e-6)
    for place in ("heads last", "itself"):
        xc, kcc, vcc = x.cuda(), kc.cuda(), vc.cuda()
        qc = xc[:, :, :Hq].transpose(1, 2)
        out = qc if place == "itself" else torch.full((B, N, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        got = E.kv_append(xc[:, :, Hq:Hq + Hk].transpose(1, 2), xc[:, :, Hq + Hk:].transpose(1, 2), kcc, vcc, table.cuda(),
                          torch.tensor(starts, dtype=torch.int32).cuda(), position_offset=5, positions=pos.cuda(),
                          inv_freq=freqs, eps=1e-6, q=qc, q_out=out)
        assert got.data_ptr() == out.data_ptr()
        O.check("k_cache", kcc, want_k, kb)
        O.check("v_cache", vcc, want_v, torch.zeros_like(want_v))
        O.check("q", out, *want_q)
        assert torch.equal(xc[:, :, Hq:].cpu(), x[:, :, Hq:]), "keys and values beside the queries stay"


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_infinity_stays_in_its_channel(E, interleaved):  # noqa: F811
    """An infinity in a channel that is not rotated reaches no other one, forward and back;
    in a rotated one it reaches its pair and nothing else."""
    q, g = rnd(170, 1, 3, 5, 64), rnd(171, 1, 3, 5, 64)
    pos, freqs = 1 + torch.arange(5)[None], E.rope_freqs(32)
    inf = float("inf")
    for at, reached in ((40, {40}), (63, {63}), (32, {32}), (3, {3, 2} if interleaved else {3, 19})):
        x, dy = q.clone(), g.clone()
        x[0, 1, 2, at] = dy[0, 1, 2, at] = inf
        xc = x.cuda().requires_grad_()
        y, _ = E.qk_norm_rope(xc, None, inv_freq=freqs, position_offset=1, interleaved=interleaved, eps=None)
        (dx,) = torch.autograd.grad(y, xc, dy.cuda())
        rest = torch.ones(64, dtype=torch.bool)
        rest[list(reached)] = False
        x0, dy0 = x.clone(), dy.clone()
        x0[0, 1, 2, at] = dy0[0, 1, 2, at] = 0.0
        for name, have, (ref, bound) in (("y", y, O.norm_rope(x0, None, pos, freqs.cpu(), interleaved, None)),
                                         ("dx", dx, O.norm_rope_back(x0, None, dy0, pos, freqs.cpu(), interleaved, None)[:2])):
            have = have.detach().cpu()
            assert not bool(torch.isfinite(have[0, 1, 2][~rest]).any())
            O.check(name, have[..., rest], ref[..., rest], bound[..., rest])
            have[0, 1, 2] = 0
            ref[0, 1, 2], bound[0, 1, 2] = 0, 0
            O.check(name + " of other rows", have, ref, bound)


def test_gradient_options_by_value(E):  # noqa: F811
    """eps and the offset given as tensors are read once, in the forward call."""
    q, g = rnd(180, 1, 2, 9, 32), rnd(181, 1, 2, 9, 32)
    eps, off = torch.tensor(0.5), torch.tensor(3)
    x = q.cuda().requires_grad_()
    f = E.rope_freqs(32)
    y, _ = E.qk_norm_rope(x, None, inv_freq=f, eps=eps, position_offset=off)
    eps.fill_(100.0)
    off.fill_(70)
    (dx,) = torch.autograd.grad(y, x, g.cuda())
    pos = 3 + torch.arange(9)[None]
    O.check("y", y, *O.norm_rope(q, None, pos, f.cpu(), False, 0.5))
    O.check("dx", dx, *O.norm_rope_back(q, None, g, pos, f.cpu(), False, 0.5)[:2])


def test_weight_gradients_by_pairs(E):  # noqa: F811
    """weight_grads: one for both, or a tuple or list of two."""
    q, k, gq, gk = (rnd(190 + i, 1, h, 9, 32).cuda() for i, h in enumerate((2, 1, 2, 1)))
    w = weight(194, 32, torch.float32).cuda()
    f = E.rope_freqs(32)
    both = E.qk_norm_rope_bwd(q, k, gq, gk, w, w, inv_freq=f)
    for how in (True, False, (True, False), [False, True], [False, False], (1, 1)):
        want = how if isinstance(how, (tuple, list)) else (how, how)
        got = E.qk_norm_rope_bwd(q, k, gq, gk, w, w, inv_freq=f, weight_grads=how)
        assert torch.equal(got[0], both[0]) and torch.equal(got[1], both[1])
        for g, b, n in zip(got[2:], both[2:], want):
            assert torch.equal(g, b) if n else g is None
