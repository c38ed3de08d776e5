"""The row operators' calls whose arguments the binding has to tell apart: empty batches."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [40, 32768])
def test_an_empty_batch(vocab):
    """Tensors without rows, whose addresses are NULL: every call is done at once and writes nothing
    but a gradient that has no terms."""
    require_gpu()
    p, h = 2, 24

    def none(n, dtype=torch.float32):
        return torch.empty((0, n), dtype=dtype, device="cuda")
    ids, empty = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    logits = [none(vocab // p) for _ in range(p)]
    print(f"[case] no tokens, vocab={vocab}", flush=True)
    B.ra_cross_entropy(logits, ids, loss=empty, lse=empty.clone())
    B.ra_cross_entropy(logits, ids, loss=empty)
    B.ra_cross_entropy(logits, ids, loss=empty, grads=logits, dloss=empty.clone())
    B.ra_cross_entropy_backward(logits, ids, empty, logits)
    tables = [torch.ones((vocab // p, h), device="cuda") for _ in range(p)]
    B.ra_embedding(tables, ids, [none(h)])
    B.ra_embedding_backward(none(h), ids, tables, accumulate=True)
    assert all(bool((t == 1).all()) for t in tables)
    B.ra_embedding_backward(none(h), ids, tables)
    assert all(bool((t == 0).all()) for t in tables)
    w = torch.ones(h, device="cuda")
    B.ra_allreduce_rmsnorm([none(h), none(h)], w, 1e-5, [none(h)], residual=none(h), residual_out=none(h), rstd=empty)
    dw = torch.ones(h, device="cuda")
    B.ra_allreduce_rmsnorm_backward([none(h)], none(h), empty, w, none(h), dh_in=none(h), dxs=[none(h)], dweight=dw)
    assert bool((dw == 0).all())
    torch.cuda.synchronize()
