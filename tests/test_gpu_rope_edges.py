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
