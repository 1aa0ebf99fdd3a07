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
