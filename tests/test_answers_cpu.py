"""Host side of the log probabilities and of the gradients' norm and clipping: argument checks,
workspace sizes and the binding's marshalling.  No call here reaches a kernel."""

import array
import ctypes

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests.test_rows_cpu import ALI, BF16, F8, F16, F32, INV, MIS, MiB, UNS, at, call

# 64 x 4096 bfloat16 logits over 2 ranks: 256 KiB a piece
LOGP = dict(logits=[at(0), at(1)], p=2, tokens=64, vocab=4096, valid=4096, dtype=BF16, scale=1.0, ids=at(2),
            id_dtype=B.RA_INT64, logprob=at(3), entropy=at(4), lse=at(5), top=20, top_ids=at(6), top_logprobs=at(7),
            ws=at(8), ws_bytes=MiB, stream=None)
VOCAB_REFUSED = [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(tokens=-1), INV), (dict(vocab=0), INV), (dict(vocab=(1 << 24) + 1), UNS),
    (dict(valid=0), INV), (dict(valid=4097), INV), (dict(dtype=B.RA_FLOAT64), UNS), (dict(dtype=F8), UNS), (dict(dtype=-1), INV),
    (dict(tokens=1 << 58), INV), (dict(id_dtype=F32), INV), (dict(logits=None), INV), (dict(logits=[at(0), 0]), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV),
    (dict(logits=[at(0), at(1) + 1]), MIS), (dict(ids=at(2) + 4), MIS), (dict(ids=None), INV),
]
SPLIT = dict(tokens=8, vocab=65536, valid=65536)      # few tokens of many columns: the call takes workspace


@pytest.mark.parametrize("change,code", VOCAB_REFUSED + [
    (dict(top=-1), INV), (dict(top=65), UNS), (dict(valid=19), INV), (dict(top_ids=None, top_logprobs=None), INV),
    (dict(logprob=None, entropy=None, lse=None, top=0), INV), (dict(logprob=at(3) + 2), MIS), (dict(top_ids=at(6) + 4), MIS),
    (dict(logprob=at(4)), ALI), (dict(lse=at(0)), ALI), (dict(top_ids=at(2)), ALI), (dict(top_logprobs=at(6) + 64), ALI),
    (dict(entropy=at(2)), ALI), (dict(top_ids=at(1) + 16), ALI),
    (dict(SPLIT, ws=None), INV), (dict(SPLIT, ws_bytes=100), INV), (dict(SPLIT, ws=at(8) + 8), MIS), (dict(SPLIT, ws=at(7)), ALI),
])
def test_logprobs_refusals(change, code):
    assert call("ra_token_logprobs", LOGP, **change) == code
    assert B.ra_last_error()


def test_logprobs_without_tokens():
    assert call("ra_token_logprobs", LOGP, tokens=0) == B.RA_OK
    none = dict(ids=None, logprob=None, entropy=None, lse=None, top_ids=None, top_logprobs=None, ws=None, ws_bytes=0)
    assert call("ra_token_logprobs", LOGP, tokens=0, **none) == B.RA_OK
    assert call("ra_token_logprobs", LOGP, tokens=0, scale=0.0) == INV


LOGPB = dict(logits=[at(0), at(1)], p=2, tokens=64, vocab=4096, valid=4096, dtype=BF16, scale=1.0, ids=at(2),
             id_dtype=B.RA_INT64, lse=at(3), entropy=at(4), dlogprob=at(5), dentropy=at(6), grads=[at(7), at(8)], stream=None)


@pytest.mark.parametrize("change,code", VOCAB_REFUSED + [
    (dict(grads=None), INV), (dict(grads=[at(7), 0]), INV), (dict(lse=None), INV), (dict(entropy=None), INV),
    (dict(dlogprob=None, dentropy=None), INV), (dict(grads=[at(1), at(0)]), ALI), (dict(grads=[at(0) + 16, at(8)]), ALI),
    (dict(grads=[at(7), at(7)]), ALI), (dict(dlogprob=at(7)), ALI), (dict(lse=at(8)), ALI), (dict(grads=[at(7), at(8) + 1]), MIS),
    (dict(dentropy=at(6) + 1), MIS),
])
def test_logprobs_backward_refusals(change, code):
    assert call("ra_token_logprobs_backward", LOGPB, **change) == code


def test_logprobs_backward_without_tokens():
    assert call("ra_token_logprobs_backward", LOGPB, tokens=0, lse=None, dlogprob=None, dentropy=None) == B.RA_OK


def test_logprobs_workspace():
    f = B.ra_token_logprobs_workspace
    assert f(0, 128000, 8, 20) == 0 and f(4096, 131072, 8, 20) == 0 and f(1, 4096, 8, 64) == 0
    one = f(1, 128000, 8, 20)
    assert 0 < one <= 64 * (16 + 8 * 20) and one % 16 == 0
    # the longest rows are always shared
    assert 0 < f(1 << 20, 1 << 24, 1, 64) <= (1 << 20) * 64 * (16 + 8 * 64)
    for p in range(1, 65):
        for v in (1 << 24, (1 << 24) - 1, 294_912, 294_913):
            assert f(1, v, p, 0) <= 64 * 16              # at most 64 parts
    for bad in ((-1, 8, 1, 0), (1, 0, 1, 0), (1, 8, 0, 0), (1, 8, 65, 0), (1, 8, 1, 9), (1, 8, 1, -1), (1, 128, 1, 65)):
        with pytest.raises(B.RaError):
            f(*bad)


def lists(sizes, codes, first=0):
    """Host arrays for a list of tensors, MiB apart."""
    return (array.array("Q", [at(first + i) if n else 0 for i, n in enumerate(sizes)]), array.array("q", sizes),
            array.array("i", codes))


def address(a):
    return a.buffer_info()[0]


WS = 16 + 8192


def grad_call(name, sizes=(1000, 0, 7), codes=(F32, BF16, F16), ptrs=None, **kw):
    p, c, t = lists(list(sizes), list(codes))
    if ptrs is not None:
        p = array.array("Q", ptrs)
    o = kw.pop("outs", None)
    o = None if o is None else array.array("Q", o)
    oc = kw.pop("out_codes", None)
    oc = None if oc is None else array.array("i", oc)
    args = dict(tensors=address(p), counts=address(c), types=address(t), n=len(sizes))
    if name == "ra_grad_clip":
        args |= dict(counted=kw.pop("counted", len(sizes)), max_norm=kw.pop("max_norm", 1.0))
    args["scale"] = 1.0
    if name == "ra_grad_clip":
        args |= dict(outs=None if o is None else address(o), out_codes=None if oc is None else address(oc))
    args |= dict(norm=at(20), ws=at(21), ws_bytes=WS, stream=None)
    args |= kw
    return getattr(B.lib(), name)(*args.values())


@pytest.mark.parametrize("name", ["ra_grad_norm", "ra_grad_clip"])
@pytest.mark.parametrize("change,code", [
    (dict(n=-1), INV), (dict(n=(1 << 20) + 1), UNS), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(tensors=None), INV), (dict(counts=None), INV), (dict(types=None), INV), (dict(sizes=(1, -1, 2)), INV),
    (dict(sizes=(1, (1 << 40) + 1, 2)), UNS), (dict(sizes=(1 << 39, 1 << 39, 1)), UNS), (dict(sizes=(1, 1 << 62, 1 << 62)), UNS),
    (dict(codes=(F32, F8, F16)), UNS),
    (dict(codes=(F32, B.RA_FLOAT64, F16)), UNS), (dict(codes=(F32, 99, F16)), INV), (dict(codes=(F32, -1, F16)), INV),
    (dict(ptrs=[at(0), 0, 0]), INV), (dict(ptrs=[at(0) + 2, 0, at(2)]), MIS), (dict(ptrs=[at(0), 0, at(2) + 1]), MIS),
    (dict(norm=None), INV), (dict(norm=at(20) + 2), MIS), (dict(norm=at(0) + 16), ALI), (dict(ws=None), INV),
    (dict(ws_bytes=WS - 1), INV), (dict(ws=at(21) + 8), MIS), (dict(ws=at(2)), ALI), (dict(ws=at(20)), ALI),
])
def test_list_refusals(name, change, code):
    assert grad_call(name, **change) == code
    assert B.ra_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(counted=-1), INV), (dict(counted=4), INV), (dict(max_norm=0.0), INV), (dict(max_norm=-1.0), INV),
    (dict(max_norm=float("nan")), INV), (dict(ptrs=[at(0), 0, at(0) + 16]), ALI), (dict(ptrs=[at(2), 0, at(2)]), ALI),
    (dict(outs=[at(10), 0, 0]), INV), (dict(outs=[at(10), 0, at(10)]), ALI), (dict(outs=[at(0) + 16, 0, at(12)]), ALI),
    (dict(outs=[at(2), 0, at(0)]), ALI), (dict(outs=[at(10) + 2, 0, at(12)]), MIS), (dict(outs=[at(20), 0, at(12)]), ALI),
    (dict(outs=[at(10), 0, at(12)], out_codes=(F32, BF16, BF16)), UNS), (dict(outs=[at(10), 0, at(12)], out_codes=(F16, BF16, F16)), UNS),
    (dict(outs=[at(10), 0, at(2)], out_codes=(F32, F32, F32)), ALI), (dict(outs=[at(10), 0, at(12)], out_codes=(F32, 77, F16)), INV),
])
def test_clip_refusals(change, code):
    assert grad_call("ra_grad_clip", **change) == code


def test_list_sizes():
    assert B.ra_grad_norm_workspace(0) == 16 and B.ra_grad_norm_workspace(1) == B.ra_grad_norm_workspace(232) == WS
    assert B.ra_grad_norm_workspace(233) == 16 + 2 * 8192
    for bad in (-1, (1 << 20) + 1):
        with pytest.raises(B.RaError):
            B.ra_grad_norm_workspace(bad)
    f = B.ra_allreduce_clip_workspace
    assert f(0) == 16 and f(1) == f(1024) == 24 and f(1025) == 32 and f(1 << 40) == 16 + 8 * 262144
    for bad in (-1, (1 << 40) + 1):
        with pytest.raises(B.RaError):
            f(bad)


FOLD = dict(bufs=[at(0), at(1)], p=2, n=1000, dtype=BF16, op=B.RA_AVG, max_norm=1.0, scale=1.0, outs=[at(2), at(3)], n_out=2,
            norm=at(4), ws=at(5), ws_bytes=24, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(n=-1), INV), (dict(n=(1 << 40) + 1), UNS), (dict(dtype=B.RA_INT32), UNS), (dict(dtype=B.RA_FLOAT64), UNS),
    (dict(dtype=50), INV), (dict(op=B.RA_MAX), UNS), (dict(op=7), INV), (dict(op=-1), INV), (dict(max_norm=0.0), INV),
    (dict(max_norm=float("nan")), INV), (dict(scale=-2.0), INV), (dict(n_out=0), INV), (dict(n_out=3), INV), (dict(bufs=None), INV),
    (dict(bufs=[at(0), 0]), INV), (dict(outs=None), INV), (dict(outs=[at(2), 0]), INV), (dict(norm=None), INV), (dict(ws=None), INV),
    (dict(ws_bytes=23), INV), (dict(ws=at(5) + 4), MIS), (dict(bufs=[at(0) + 1, at(1)]), MIS), (dict(norm=at(4) + 1), MIS),
    (dict(bufs=[at(0), at(0)], outs=[at(0), at(3)]), ALI), (dict(outs=[at(2), at(2)]), ALI), (dict(outs=[at(0) + 16, at(3)]), ALI),
    (dict(outs=[at(0), at(0)]), ALI), (dict(norm=at(2)), ALI), (dict(ws=at(3)), ALI), (dict(ws=at(4)), ALI),
])
def test_allreduce_clip_refusals(change, code):
    assert call("ra_allreduce_clip", FOLD, **change) == code
    assert B.ra_last_error()


def test_binding_wants_device_tensors():
    x = [torch.zeros(4, 8)]
    norm = torch.zeros(1)
    with pytest.raises(ValueError, match="device tensors"):
        B.ra_token_logprobs(x, lse=torch.zeros(4))
    with pytest.raises(ValueError, match="device tensors"):
        B.ra_token_logprobs_backward(x, torch.zeros(4, dtype=torch.int64), norm, x, dlogprob=norm)
    with pytest.raises(ValueError):
        B.TensorList([norm])
    with pytest.raises(ValueError, match="device tensor"):
        B.ra_grad_norm([], norm)
    with pytest.raises(ValueError):
        B.ra_grad_clip([norm], 1.0, norm)
    with pytest.raises(ValueError, match="device tensors"):
        B.ra_allreduce_clip([norm], 1.0, norm)


def test_forms_in_64_bits():
    """The reference's gradient against autograd, its best columns by hand."""
    from tests import answers_ref as A
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, 40), generator=g)
    y = torch.tensor([0, 39, 7, 7, 20])
    da, db = torch.randn(5, generator=g), torch.randn(5, generator=g)
    z = x.double().requires_grad_()
    ln_p = torch.log_softmax(z * 0.5, 1)
    ((da * ln_p.gather(1, y.unsqueeze(1)).squeeze(1)).sum() - (db.unsqueeze(1) * ln_p.exp() * ln_p).sum()).backward()
    (lp, ent, lse, cols, top), _ = A.logprobs(x, y, 0.5, 40, 3)
    d, err = A.logprobs_backward(x, y, lse, ent, da, db, 0.5, 40)
    assert (d - z.grad).abs().max() < 1e-12 and (err > 0).all() and err.max() < 1e-5
    assert torch.allclose(lp, ln_p.gather(1, y.unsqueeze(1)).squeeze(1).detach())
    assert torch.equal(cols, torch.topk(x, 3).indices)
    rows = torch.tensor([[1.0, 2.0, 2.0, float("nan"), -0.0, 0.0], [float("-inf")] * 6])
    assert A.best(rows, 4).tolist() == [[3, 1, 2, 0], [0, 1, 2, 3]]
    assert A.best(rows[:, 4:], 2).tolist() == [[0, 1], [0, 1]]
    n, _ = A.norm([torch.tensor([3.0]), torch.tensor([4.0])], 2.0)
    assert n == 10.0 and abs(A.factor(n, 5.0, 2.0)[0] - 1.0) < 1e-6
    assert ctypes.sizeof(ctypes.c_void_p) == 8
