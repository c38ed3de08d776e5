"""The row operators' calls whose arguments the binding has to tell apart: empty batches, rows
of another length, and RankBuffers in place of lists."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
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


def shaped(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype, device="cuda")


def test_rows_of_another_length_are_refused():
    """As many elements, but not in rows of the weight's or the table's length."""
    require_gpu()
    w8, r8, ids4 = shaped(8), shaped(8), torch.zeros(4, dtype=torch.int64, device="cuda")

    def norm(bufs, weight=w8, outs=None, **kw):
        B.ra_allreduce_rmsnorm(bufs, weight, 1e-5, outs or [shaped(8, 8)], **kw)

    def back(dys, h, dh, **kw):
        B.ra_allreduce_rmsnorm_backward(dys, h, r8, w8, dh, **kw)
    wide, fit = (lambda: shaped(4, 16)), (lambda: shaped(8, 8))
    for refused in (lambda: norm([wide()]), lambda: norm([wide(), wide()], outs=[wide()]),
                    lambda: norm([fit(), wide()]), lambda: norm(B.RankBuffers([wide()])),
                    lambda: norm(B.RankBuffers([fit(), wide()])), lambda: norm([shaped(4, 1, 16)]),
                    lambda: norm([fit()], outs=[wide()]), lambda: norm([fit()], outs=[fit(), wide()]),
                    lambda: norm([fit(), fit()], outs=B.RankBuffers([wide(), wide()])),
                    lambda: norm([fit()], residual=wide()), lambda: norm([fit()], residual_out=wide()),
                    lambda: norm([shaped(64)], outs=[wide()]),
                    lambda: back([wide()], fit(), fit()), lambda: back([fit()], wide(), fit()),
                    lambda: back([fit()], fit(), wide()), lambda: back([fit()], fit(), fit(), dh_in=wide()),
                    lambda: back([fit()], fit(), fit(), dxs=[wide()]),
                    lambda: B.ra_embedding([shaped(5, 8)], ids4, [shaped(2, 16)]),
                    lambda: B.ra_embedding([shaped(3, 8), shaped(2, 8)], ids4, [shaped(4, 8), shaped(2, 16)]),
                    lambda: B.ra_embedding_backward(shaped(2, 16), ids4, [shaped(5, 8)])):
        with pytest.raises(ValueError, match="rows of 8"):
            refused()
    torch.cuda.synchronize()


def test_rows_with_several_leading_dimensions_and_flat_ones():
    """What counts is the last dimension: [2, 4, 8] is [8, 8], and a flat array has its rows one
    behind the other."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(12)
    x, res, w = [torch.randn((2, 8, 8), device="cuda", generator=g) for _ in range(2)] + [shaped(8)]
    want, wide = shaped(8, 8), shaped(8, 8)
    B.ra_allreduce_rmsnorm(list(x.unbind(0)), w, 1e-5, [want], residual=res[0], residual_out=wide)
    for shape in ((8, 8), (2, 4, 8), (8, 1, 8), (64,)):
        y, h = shaped(*shape), shaped(*shape)
        bufs = [b.view(shape) for b in x.unbind(0)]
        B.ra_allreduce_rmsnorm(bufs, w, 1e-5, [y], residual=res[0].view(shape), residual_out=h)
        assert torch.equal(y.view(8, 8), want) and torch.equal(h.view(8, 8), wide)
        y.fill_(0)
        B.ra_allreduce_rmsnorm(B.RankBuffers([bufs[0], bufs[1].view(8, 8)]), w, 1e-5, [y], residual=res[0])
        assert torch.equal(y.view(8, 8), want)
        ids = torch.tensor([0, 3, 3, 1, 4, 2, 0, 1], device="cuda")
        table, rows, d = torch.randn((5, 8), device="cuda", generator=g), shaped(*shape), shaped(5, 8)
        B.ra_embedding([table], ids, [rows])
        assert torch.equal(rows.view(8, 8), table[ids])
        B.ra_embedding_backward(rows, ids, [d])
        want_d, err, _ = R.embedding_backward(rows.view(8, 8), ids, 5, 1.0, None)
        R.check(d, want_d, R.rounded(want_d, err, torch.float32), "dtable")


def test_rank_buffers_of_8_bit_outputs_and_their_scales():
    """A RankBuffers in place of every list of the 8-bit call; other calls refuse such outputs."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(13)
    bufs, w = [torch.randn((6, 48), device="cuda", generator=g) for _ in range(3)], shaped(48)
    for group in (0, 32):
        def run(wrap):
            outs = [torch.zeros((6, 48), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(3)]
            scales = [torch.zeros((6, 2 if group else 1), device="cuda") for _ in range(3)]
            B.ra_allreduce_rmsnorm(wrap(bufs), w, 1e-5, wrap(outs), scales=wrap(scales), group=group)
            return [o.view(torch.uint8) for o in outs] + scales
        lists, wrapped = run(list), run(B.RankBuffers)
        assert all(torch.equal(a, b) for a, b in zip(lists, wrapped)) and bool((wrapped[-1] > 0).all())
    eight = B.RankBuffers([torch.zeros((6, 48), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(3)])
    for refused in (lambda: B.ra_allreduce(eight), lambda: B.ra_allreduce_ex(eight, algo="tree"),
                    lambda: B.ra_reduce_scatter(eight), lambda: B.ra_all_gather(eight),
                    lambda: B.ra_allreduce_noalloc(eight), lambda: B.ra_allreduce_rmsnorm(eight, w, 1e-5, bufs)):
        with pytest.raises((B.RaError, TypeError)):
            refused()
    with pytest.raises(TypeError):
        B.ra_allreduce(list(eight.tensors))
    torch.cuda.synchronize()
