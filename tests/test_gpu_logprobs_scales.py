"""ra_token_logprobs and its backward at the largest scales that there are: scale log2 e is beyond
float32, the log probabilities are not."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import answers_ref as A
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.pads import cut

pytestmark = pytest.mark.gpu

LARGEST = 3.4028234663852886e38


@pytest.mark.parametrize("scale", [2.3e38, 2.4e38, LARGEST])
@pytest.mark.parametrize("p,t,v", [(4, 3, 60_000), (4, 150, 5000), (1, 20, 300), (3, 7, 20)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -127])
def test_largest_scales(scale, p, t, v, size):
    """Logits of some 1 (all of a row's probability is in its largest ones) and of some 1 / scale."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(t + v)
    # whole numbers of sixteenths, scaled exactly; below 2^-126 as well
    x = (16 * torch.randn((t, v), device="cuda", generator=g)).round() / 16 * size
    x[0, v // 3] = -torch.inf
    x[1] = -x[1].abs()                                        # a largest logit of 0 or below
    x[2] = -x[2].abs() - size
    y = torch.randint(0, v, (t,), device="cuda", generator=g)
    y[::2] = x.argmax(1)[::2]
    lp, ent, lse = (torch.empty(t, device="cuda") for _ in range(3))
    ids, tlp = torch.empty((t, 5), dtype=torch.int64, device="cuda"), torch.empty((t, 5), device="cuda")
    print(f"[case] scale {scale} p={p} t={t} v={v} size {size}", flush=True)
    B.ra_token_logprobs(cut(x, p), y, lp, ent, lse, ids, tlp, scale=scale)
    want, err = A.logprobs(x, y, scale, v, 5)
    assert torch.equal(ids, want[3])
    for got, w, e, what in ((lp, want[0], err[0], "logprob"), (ent, want[1], err[1], "entropy"),
                            (lse, want[2], err[2], "lse"), (tlp, want[4], err[4], "top_logprobs")):
        R.check(got, w, R.rounded(torch.where(w.isfinite(), w, 0.0), e, torch.float32), what)
    if size == 1.0:
        return
    da, db = torch.full((t,), 2.0 ** -100, device="cuda"), torch.full((t,), -2.0 ** -104, device="cuda")
    grads = [torch.empty_like(c) for c in cut(x, p)]
    B.ra_token_logprobs_backward(cut(x, p), y, lse, grads, da, ent, db, scale=scale)
    d, e = A.logprobs_backward(x, y, lse, ent, da, db, scale, v)
    R.check(torch.cat(grads, 1), d, R.rounded(d, e, torch.float32), "grads")


@pytest.mark.parametrize("scale", [1e-39, 1.2e-38, 5e-38, 1e-36, 1e-30, 1.0, 1e10])
@pytest.mark.parametrize("p,t,v", [(4, 3, 60_000), (4, 150, 5000), (1, 20, 300), (3, 7, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_at_both_ends(scale, p, t, v, dtype):
    """Differences of logits are beyond float32, and scale times them are not always."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(t + v)
    x = ((2 * torch.rand((t, v), device="cuda", generator=g) - 1) * 3.3e38).to(dtype)
    x[0, v // 2:] = -torch.inf
    x[1, :v // 2] = -3.3e38                                   # whole parts of a row far below the others
    x[2, v // 2:] = -3.3e38
    x[2, v // 2 + 1] = 3.3e38
    y = torch.randint(0, v, (t,), device="cuda", generator=g)
    lp, ent, lse = (torch.empty(t, device="cuda") for _ in range(3))
    ids, tlp = torch.empty((t, 9), dtype=torch.int64, device="cuda"), torch.empty((t, 9), device="cuda")
    print(f"[case] ends scale {scale} p={p} t={t} v={v} {dtype}", flush=True)
    B.ra_token_logprobs(cut(x, p), y, lp, ent, lse, ids, tlp, scale=scale)
    want, err = A.logprobs(x, y, scale, v, 9)
    assert torch.equal(ids, want[3])
    for got, w, e, what in ((lp, want[0], err[0], "logprob"), (ent, want[1], err[1], "entropy"),
                            (lse, want[2], err[2], "lse"), (tlp, want[4], err[4], "top_logprobs")):
        R.check(got, w, R.rounded(torch.where(w.isfinite(), w, 0.0), e, torch.float32), what)
