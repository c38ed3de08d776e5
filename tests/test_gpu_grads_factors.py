"""Clipping of gradients near float32's end by norms near its other end: the factor is far below what
float32 has, the clipped gradients are not."""

import math

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


# factors of 2^-129 to 2^-248; the clipped gradients are normal numbers of float32
@pytest.mark.parametrize("max_norm", [10.0, 1e-20, 1e-25, 1e-27, 1e-28, 1e-30, 1e-33, 1e-35])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_factors_of_large_gradients(max_norm, dtype):
    require_gpu()
    x = torch.tensor([2e38, -1.5e38, 2.5e38, 3e37], device="cuda").repeat(250).to(dtype)
    m = float(torch.tensor(max_norm, dtype=torch.float32))
    n = math.sqrt(float((x.double() ** 2).sum()))
    c = m / (n + 1e-6)
    # the factor, and two products, are rounded to float32 once each
    want = x.double() * c
    tol = 3 * R.U * want.abs()
    norm, out = torch.empty(1, device="cuda"), torch.empty(1000, device="cuda")
    B.ra_grad_clip([x], max_norm, norm, outs=[out])
    assert norm.item() == math.inf                       # beyond float32
    R.check(out, want, tol, "clipped into float32")
    if dtype is torch.bfloat16:
        B.ra_allreduce_clip([x, torch.zeros_like(x)], max_norm, norm, op="sum")
        R.check(x, want, R.rounded(want, tol, dtype), "summed and clipped")
    else:
        B.ra_grad_clip([x], max_norm, norm)
        R.check(x, want, tol, "clipped in place")


def test_a_factor_of_zero():
    """Of an infinite norm: what is finite becomes zero."""
    require_gpu()
    x, norm = torch.tensor([1.0, math.inf, -3e38], device="cuda"), torch.empty(1, device="cuda")
    out = torch.full((3,), 7.0, device="cuda")
    B.ra_grad_clip([x], 1.0, norm, outs=[out])
    assert norm.item() == math.inf and out[0] == 0 and out[2] == 0 and out[1].isnan()
