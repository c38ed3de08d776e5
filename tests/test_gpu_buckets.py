"""Gradients in several buckets on every rank: each bucket all-reduced, then all of them clipped by one norm,
rank 0's buckets being the counted ones; against 64 bits."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import answers_ref as A
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.pads import padded, untouched

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p", [2, 5])
def test_buckets_clipped_by_one_norm(p, dtype):
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(p)
    buckets = [[padded((n,), dtype, 8, torch.randn(n, device="cuda", generator=g).to(dtype)) for _ in range(p)]
               for n in (1000, 33, 70_001, 1)]
    for b in buckets:
        B.ra_allreduce(b, op="avg")
    sums = [b[0].clone() for b in buckets]
    tensors = [b[r] for r in range(p) for b in buckets]
    norm = torch.empty(1, device="cuda")
    print(f"[case] buckets p={p} {dtype}", flush=True)
    B.ra_grad_clip(tensors, 0.5, norm, counted=len(buckets))
    want, err = A.norm(sums, 1.0)
    assert abs(float(norm.double()) - want) <= err and want > 0.5
    c, ec = A.factor(want, 0.5, 1.0)
    for b, s in zip(buckets, sums):
        d, tol = A.scaled(s, c, ec, dtype)
        for x in b:
            R.check(x, d, tol, "clipped")
            untouched(x)
