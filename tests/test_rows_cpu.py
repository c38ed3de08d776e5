"""Host side of the row operators (norm, cross entropy, embedding): argument checks,
workspace sizes and the binding's marshalling.  No call here reaches a kernel."""

import ctypes

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B

MiB = 1 << 20
BASE = 0x7f0000000000
INV, UNS, ALI, MIS = B.RA_ERR_INVALID_ARG, B.RA_ERR_UNSUPPORTED, B.RA_ERR_ALIAS, B.RA_ERR_MISALIGNED
F32, BF16, F16, F8 = B.RA_FLOAT32, B.RA_BFLOAT16, B.RA_FLOAT16, B.RA_FLOAT8_E4M3


def at(i):
    return BASE + i * MiB


def ptrs(addrs):
    return (ctypes.c_void_p * max(1, len(addrs)))(*addrs)


def call(name, defaults, **kw):
    args = dict(defaults, **kw)
    vals = []
    for v in args.values():
        vals.append(ptrs(v) if isinstance(v, list) else v)
    return getattr(B.lib(), name)(*vals)


# 64 x 1024 bfloat16 rows: 128 KiB an array, arrays a MiB apart.  n_out etc. are not met by
# a kernel: every call below is refused, or has no tokens.
NORM = dict(bufs=[at(0), at(1)], p=2, tokens=64, hidden=1024, dtype=BF16, res_in=at(2), res_out=at(3),
            res_dtype=BF16, weight=at(4), eps=1e-5, outs=[at(5), at(6)], n_out=2, out_dtype=BF16,
            scales=None, group=0, rstd=at(7), stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(tokens=-1), INV), (dict(hidden=0), INV), (dict(hidden=32769), UNS),
    (dict(tokens=1 << 58), INV), (dict(dtype=9), INV), (dict(dtype=B.RA_INT32), UNS), (dict(dtype=B.RA_FLOAT64), UNS),
    (dict(dtype=F8), UNS), (dict(res_dtype=F16), UNS), (dict(res_dtype=77), INV), (dict(out_dtype=F32), UNS),
    (dict(out_dtype=99), INV), (dict(n_out=0), INV), (dict(n_out=3), INV), (dict(group=16), INV), (dict(group=32), INV),
    (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(bufs=None), INV), (dict(bufs=[at(0), 0]), INV), (dict(weight=None), INV), (dict(outs=None), INV),
    (dict(outs=[at(5), 0]), INV), (dict(out_dtype=F8), INV), (dict(out_dtype=F8, scales=[at(8), 0]), INV),
    (dict(bufs=[at(0) + 1, at(1)]), MIS), (dict(weight=at(4) + 1), MIS), (dict(rstd=at(7) + 2), MIS),
    (dict(res_dtype=F32, res_in=at(2) + 2), MIS), (dict(outs=[at(5), at(6) + 1]), MIS),
    (dict(outs=[at(5), at(5)]), ALI), (dict(outs=[at(0), at(0)]), ALI), (dict(outs=[at(0) + 16, at(6)]), ALI),
    (dict(outs=[at(4), at(6)]), ALI), (dict(res_out=at(0)), ALI), (dict(res_out=at(2) + 16), ALI),
    (dict(rstd=at(5) + 64), ALI), (dict(out_dtype=F8, outs=[at(0), at(6)], scales=[at(8), at(9)]), ALI),
    (dict(out_dtype=F8, scales=[at(8), at(8)]), ALI), (dict(res_dtype=F32, res_out=at(4) - 64), ALI),
])
def test_norm_refusals(change, code):
    assert call("ra_allreduce_rmsnorm", NORM, **change) == code
    assert B.ra_last_error()


def test_norm_without_tokens():
    assert call("ra_allreduce_rmsnorm", NORM, tokens=0) == B.RA_OK
    assert call("ra_allreduce_rmsnorm", NORM, tokens=0, eps=0.0) == INV


BWD = dict(dys=[at(0), at(1)], p=2, tokens=64, hidden=1024, dtype=BF16, h=at(2), h_dtype=F32, rstd=at(3),
           weight=at(4), dh_in=at(5), dh=at(6), dxs=[at(7)], n_dx=1, dweight=at(8), ws=at(9), ws_bytes=64 * 4096,
           stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(hidden=32769), UNS), (dict(tokens=-2), INV), (dict(dtype=B.RA_INT64), UNS),
    (dict(h_dtype=F16), UNS), (dict(n_dx=-1), INV), (dict(n_dx=3), INV), (dict(dys=None), INV), (dict(h=None), INV),
    (dict(rstd=None), INV), (dict(weight=None), INV), (dict(dh=None), INV), (dict(dxs=None), INV), (dict(dxs=[0]), INV),
    (dict(ws=None), INV), (dict(ws_bytes=64 * 4096 - 1), INV), (dict(ws=at(9) + 4), MIS), (dict(h=at(2) + 2), MIS),
    (dict(dweight=at(8) + 1), MIS), (dict(dh=at(2)), ALI), (dict(dh=at(5) + 16), ALI), (dict(dxs=[at(0) + 32]), ALI),
    (dict(dxs=[at(6)]), ALI), (dict(dweight=at(4)), ALI), (dict(ws=at(8)), ALI), (dict(dxs=[at(0), at(0)], n_dx=2), ALI),
])
def test_norm_backward_refusals(change, code):
    assert call("ra_allreduce_rmsnorm_backward", BWD, **change) == code


def test_norm_backward_without_tokens():
    assert call("ra_allreduce_rmsnorm_backward", BWD, tokens=0, dweight=None, ws=None, ws_bytes=0) == B.RA_OK


# 64 x 4096 bfloat16 logits over 2 ranks: 256 KiB a piece
XENT = dict(logits=[at(0), at(1)], p=2, tokens=64, vocab=4096, valid=4096, dtype=BF16, targets=at(2),
            target_dtype=B.RA_INT64, loss=at(3), lse=at(4), grads=[at(5), at(6)], dloss=at(7), scale=1.0,
            ws=at(8), ws_bytes=MiB, stream=None)
XENT_REFUSED = [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(tokens=-1), INV), (dict(vocab=0), INV), (dict(vocab=(1 << 24) + 1), UNS),
    (dict(valid=0), INV), (dict(valid=4097), INV), (dict(dtype=B.RA_FLOAT64), UNS), (dict(dtype=-1), INV),
    (dict(target_dtype=F32), INV), (dict(logits=None), INV), (dict(logits=[at(0), 0]), INV), (dict(targets=None), INV),
    (dict(grads=[at(5), 0]), INV), (dict(logits=[at(0), at(1) + 1]), MIS), (dict(targets=at(2) + 4), MIS),
    (dict(grads=[at(1), at(0)]), ALI), (dict(grads=[at(0) + 16, at(6)]), ALI), (dict(grads=[at(5), at(5)]), ALI),
    (dict(dloss=at(5)), ALI),
]


# few tokens of many columns: the call takes workspace
SPLIT = dict(tokens=8, vocab=32768, valid=32768)


@pytest.mark.parametrize("change,code", XENT_REFUSED + [
    (dict(loss=None, lse=None, grads=None), INV), (dict(loss=at(2)), ALI), (dict(loss=at(4)), ALI),
    (dict(lse=at(0)), ALI),
    (dict(SPLIT, ws=None), INV), (dict(SPLIT, ws_bytes=100), INV), (dict(SPLIT, ws=at(8) + 8), MIS),
    (dict(SPLIT, ws=at(5)), ALI),
])
def test_cross_entropy_refusals(change, code):
    assert call("ra_cross_entropy", XENT, **change) == code


XENT_BWD = {k: XENT[k] for k in ("logits", "p", "tokens", "vocab", "valid", "dtype", "targets", "target_dtype", "lse",
                                 "grads", "dloss", "scale", "stream")}


@pytest.mark.parametrize("change,code", XENT_REFUSED + [(dict(grads=None), INV), (dict(lse=None), INV),
                                                         (dict(lse=at(5)), ALI)])
def test_cross_entropy_backward_refusals(change, code):
    assert call("ra_cross_entropy_backward", XENT_BWD, **change) == code


def test_cross_entropy_without_tokens():
    assert call("ra_cross_entropy", XENT, tokens=0) == B.RA_OK
    assert call("ra_cross_entropy_backward", XENT_BWD, tokens=0) == B.RA_OK


EMB = dict(tables=[at(0), at(1)], p=2, vocab=1000, hidden=128, dtype=BF16, ids=at(2), id_dtype=B.RA_INT32, tokens=64,
           scale=1.0, outs=[at(3), at(4)], n_out=2, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(vocab=0), INV), (dict(vocab=(1 << 24) + 1), UNS), (dict(hidden=0), INV),
    (dict(hidden=(1 << 20) + 1), UNS), (dict(tokens=-1), INV), (dict(dtype=B.RA_INT32), UNS), (dict(id_dtype=BF16), INV),
    (dict(n_out=0), INV), (dict(n_out=3), INV), (dict(tables=None), INV), (dict(tables=[0, at(1)]), INV),
    (dict(ids=None), INV), (dict(outs=None), INV), (dict(outs=[0, at(4)]), INV), (dict(ids=at(2) + 2), MIS),
    (dict(tables=[at(0) + 1, at(1)]), MIS), (dict(outs=[at(3), at(3)]), ALI), (dict(outs=[at(0), at(4)]), ALI),
    (dict(outs=[at(3), at(2) - 16]), ALI),
])
def test_embedding_refusals(change, code):
    assert call("ra_embedding", EMB, **change) == code


EMB_BWD = dict(dy=at(0), tokens=64, hidden=128, dtype=BF16, ids=at(1), id_dtype=B.RA_INT64, scale=1.0,
               dtables=[at(2), at(3)], p=2, vocab=1000, dtable_dtype=F32, accumulate=0, ws=at(4), ws_bytes=MiB,
               stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(p=0), INV), (dict(p=65), UNS), (dict(vocab=0), INV), (dict(hidden=0), INV), (dict(tokens=-1), INV),
    (dict(tokens=1 << 31), UNS), (dict(dtype=B.RA_FLOAT64), UNS), (dict(dtable_dtype=F16), UNS), (dict(id_dtype=F16), INV),
    (dict(dy=None), INV), (dict(ids=None), INV), (dict(dtables=None), INV), (dict(dtables=[at(2), 0]), INV),
    (dict(ws=None), INV), (dict(ws_bytes=64), INV), (dict(ws=at(4) + 8), MIS), (dict(dy=at(0) + 1), MIS),
    (dict(ids=at(1) + 4), MIS), (dict(dtables=[at(2), at(2)]), ALI), (dict(dtables=[at(0), at(3)]), ALI),
    (dict(dtables=[at(1) - 16, at(3)]), ALI), (dict(ws=at(2)), ALI),
])
def test_embedding_backward_refusals(change, code):
    assert call("ra_embedding_backward", EMB_BWD, **change) == code


def test_pieces_without_columns_may_be_null():
    # 3 columns over 5 ranks: ranks 3 and 4 have none; refused for another reason (NULL targets)
    assert call("ra_cross_entropy", XENT, logits=[at(0), at(1), at(2), 0, 0], grads=None, p=5, vocab=3, valid=3,
                targets=None) == INV
    assert "targets" in B.ra_last_error()
    assert call("ra_embedding", EMB, tables=[at(0), at(1), at(2), 0, 0], p=5, vocab=3, ids=None) == INV
    assert "ids" in B.ra_last_error()


def test_workspace_sizes():
    assert B.ra_allreduce_rmsnorm_backward_workspace(0, 128) == 0
    for t in (1, 7, 512, 513, 1 << 20):
        assert B.ra_allreduce_rmsnorm_backward_workspace(t, 1000) <= 512 * 1000 * 4
        assert B.ra_allreduce_rmsnorm_backward_workspace(t, 1000) >= 4000
        assert B.ra_embedding_backward_workspace(t, 100, 64) >= 8 * t
        assert B.ra_cross_entropy_workspace(t, 128000, 8) >= 0
    assert B.ra_cross_entropy_workspace(1 << 20, 128000, 8) == 0
    assert B.ra_cross_entropy_workspace(8, 32768, 2) > 100
    for f, args in ((B.ra_allreduce_rmsnorm_backward_workspace, (-1, 8)), (B.ra_allreduce_rmsnorm_backward_workspace, (1, 0)),
                    (B.ra_cross_entropy_workspace, (1, 0, 2)), (B.ra_cross_entropy_workspace, (1, 8, 0)),
                    (B.ra_embedding_backward_workspace, (1, 5, -3)),
                    (B.ra_embedding_backward_workspace, (1, 0, 3))):
        with pytest.raises(B.RaError) as e:
            f(*args)
        assert e.value.code == INV
    lib = B.lib()
    assert lib.ra_allreduce_rmsnorm_backward_workspace(1, 8, None) == INV
    assert lib.ra_cross_entropy_workspace(1, 8, 1, None) == INV
    assert lib.ra_embedding_backward_workspace(1, 8, 8, None) == INV


def test_other_calls_do_not_take_the_8_bit_type():
    buf = ptrs([at(0), at(1)])
    assert B.lib().ra_allreduce(buf, 2, 16, F8, 0, None) == INV
    out = ctypes.c_int()
    assert B.lib().ra_select_algo(2, 16, F8, None, ctypes.byref(out)) == INV


def test_binding_refuses_host_tensors():
    x, w, ids = torch.zeros(2, 8), torch.ones(8), torch.zeros(2, dtype=torch.int64)
    for f in (lambda: B.ra_allreduce_rmsnorm([x, x], w, 1e-5, [x]),
              lambda: B.ra_allreduce_rmsnorm([], w, 1e-5, [x]),
              lambda: B.ra_allreduce_rmsnorm_backward([x], x, w, w, x),
              lambda: B.ra_cross_entropy([x], ids, loss=torch.zeros(2)),
              lambda: B.ra_cross_entropy_backward([x], ids, torch.zeros(2), [x]),
              lambda: B.ra_embedding([x], ids, [x]),
              lambda: B.ra_embedding_backward(x, ids, [x])):
        with pytest.raises(ValueError):
            f()


def test_pieces_have_to_be_cut_as_the_library_cuts_them():
    def cut(*sizes):
        return B._cut_table("t", [torch.zeros(2, n) for n in sizes], 1, 2)[1]
    assert cut(4, 3, 3) == 10 and cut(2, 2) == 4 and cut(1, 0, 0) == 1
    for sizes in ((3, 4, 3), (5, 3, 2), (4, 4, 2), (0, 1)):
        with pytest.raises(ValueError):
            cut(*sizes)
    with pytest.raises(ValueError):
        B._cut_table("t", [torch.zeros(2, 3), torch.zeros(3, 3)], 1, 2)
