"""A TensorList of which one tensor, not the first, was resized or re-pointed is refused by every call
that takes one, before anything is launched."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [1, 3])
def test_every_tensor_of_a_list_is_looked_at(which):
    require_gpu()
    n = torch.empty(1, device="cuda")

    def fresh():
        return [torch.randn(64 + i, device="cuda") for i in range(4)]
    for change in (lambda t: t.set_(torch.zeros(4096, device="cuda")[1024:1024 + t.numel()]),
                   lambda t: t.resize_(t.numel() - 1), lambda t: t.resize_(1 << 20)):
        g, other = fresh(), fresh()
        held = B.TensorList(g)
        B.ra_grad_norm(held, n)
        want = float(n)
        keep = [t.clone() for t in other]
        change(g[which])
        n.fill_(-1.0)
        for call in (lambda: B.ra_grad_norm(held, n), lambda: B.ra_grad_clip(held, 1.0, n),
                     lambda: B.ra_grad_clip(other, 1.0, n, held)):
            with pytest.raises(ValueError, match="re-pointed"):
                call()
        torch.cuda.synchronize()
        assert float(n) == -1.0 and want > 0
        assert all(torch.equal(a, b) for a, b in zip(other, keep))
        g[which].fill_(0.5)                          # memory that it got anew holds anything
        B.ra_grad_norm(B.TensorList(g), n)           # made anew
        assert torch.isfinite(n).all()
