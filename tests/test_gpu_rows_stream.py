"""The row operators' streaming kernels, which calls of more than 512 MiB with aligned rows run,
against the 64-bit forms: sizes just above that, with row counts that divide by nothing."""

import math

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.test_gpu_rows_norm import T, make, padded, untouched

pytestmark = pytest.mark.gpu

STREAMS = 512 << 20
SIZE = {"f32": 4, "bf16": 2, "f16": 2}

NORM = [
    # p, tokens, hidden, dtype, residual, group (None: not in 8 bits), outputs, in place
    (8, 3001, 8192, "bf16", "bf16", None, 1, False), (8, 1701, 8192, "bf16", "f32", None, 8, True),
    (9, 2763, 8192, "f16", "f16", None, 1, False), (3, 1401, 16384, "f32", "f32", None, 1, True),
    (4, 60001, 512, "f16", "f32", None, 1, False), (7, 70003, 520, "bf16", None, None, 1, False),
    (8, 3101, 8192, "bf16", "bf16", 0, 2, False), (8, 3101, 8192, "bf16", "bf16", 128, 2, False),
    (2, 1841, 32768, "bf16", "bf16", 32, 1, False), (5, 186007, 264, "f16", None, 64, 1, False),
    (1, 10949, 16384, "bf16", None, 0, 1, False),
]


@pytest.mark.parametrize("p,t,h,dt,rt,group,n_out,in_place", NORM)
def test_norm(p, t, h, dt, rt, group, n_out, in_place):
    require_gpu()
    f8 = group is not None
    moved = t * h * (p * SIZE[dt] + (2 * SIZE[rt] if rt else 0) + n_out * (1 if f8 else SIZE[dt]))
    assert moved > STREAMS
    bufs, g = make(p, t, h, T[dt], seed=p + t)
    residual = 3 * torch.randn((t, h), device="cuda", generator=g) if rt else None
    residual = padded((t, h), T[rt], 0, residual) if rt else (None, None)
    weight = (1 + 0.2 * torch.randn(h, device="cuda", generator=g)).to(T[dt])
    hh, r, y, eh, er, ey = R.norm(bufs, residual[0], weight, 1e-5)
    rstd = padded((t,), torch.float32)
    if in_place:
        outs, rout = [(b, None) for b in bufs[:n_out]], residual
    else:
        ot = torch.float8_e4m3fn if f8 else T[dt]
        outs = [padded((t, h), ot) for _ in range(n_out)]
        rout = padded((t, h), T[rt]) if rt else (None, None)
    groups = -(-h // group) if group else 1
    scales = [padded((t, groups), torch.float32) for _ in outs] if f8 else None
    print(f"[case] stream norm p={p} t={t} h={h} {dt} {rt} group={group} n_out={n_out} {in_place}", flush=True)
    B.ra_allreduce_rmsnorm(bufs, weight, 1e-5, [o[0] for o in outs], residual=residual[0], residual_out=rout[0],
                           scales=[s[0] for s in scales] if f8 else None, group=group or 0, rstd=rstd[0])
    R.check(rstd[0], r, er, "rstd")
    untouched(rstd[1], 0, t)
    if rt:
        R.check(rout[0], hh, R.rounded(hh, eh, T[rt]), "residual_out")
        untouched(rout[1], 0, t * h)
    for k, (o, flat) in enumerate(outs):
        if flat is not None:
            untouched(flat, 0, t * h)
        if k > 0:
            assert torch.equal(o.view(torch.uint8), outs[0][0].view(torch.uint8))
    if not f8:
        R.check(outs[0][0], y, R.rounded(y, ey, T[dt]), "y")
        return
    cols = group or h
    pad = (0, groups * cols - h)
    top = torch.nn.functional.pad(y.abs(), pad).view(t, groups, cols).amax(2)
    etop = torch.nn.functional.pad(ey, pad).view(t, groups, cols).amax(2)
    want = top.clamp_min(2.0 ** -110) / 448
    for s, flat in scales:
        R.check(s, want, etop / 448 + 2 * R.U * want, "scale")
        untouched(flat, 0, t * groups)
    sc = scales[0][0].double().repeat_interleave(cols, 1)[:, :h]
    # e4m3 is off by 2^-4 relative, and by half its smallest step (2^-10) where it is
    # subnormal; the quotient by 3 u, the product here by none
    tol = (y.abs() + ey) * (2.0 ** -4 + 3 * R.U) + ey + 2.0 ** -10 * sc
    R.check(outs[0][0].double() * sc, y, tol, "q * scale")


BACKWARD = [
    # p, tokens, hidden, dtype, h's type, copies, dh_in, in place
    (8, 2763, 8192, "bf16", "bf16", 1, True, False), (8, 2301, 8192, "bf16", "f32", 1, True, False),
    (8, 1751, 8192, "f16", "f16", 8, True, True), (4, 1501, 16384, "f16", "f32", 1, True, False),
    (2, 701, 32768, "f32", "f32", 1, True, True), (8, 50007, 512, "bf16", "bf16", 1, True, False),
    (9, 80001, 264, "bf16", "f32", 0, False, False),
]


@pytest.mark.parametrize("p,t,h,dt,ht,copies,with_dh,in_place", BACKWARD)
def test_norm_backward(p, t, h, dt, ht, copies, with_dh, in_place):
    require_gpu()
    assert t * h * (p * SIZE[dt] + (3 if with_dh else 2) * SIZE[ht] + copies * SIZE[dt]) > STREAMS
    dys, g = make(p, t, h, T[dt], seed=p + t)
    hh = (2 * torch.randn((t, h), device="cuda", generator=g)).to(T[ht])
    rstd = (hh.double().square().mean(1) + 1e-5).rsqrt().float()
    w = (1 + 0.2 * torch.randn(h, device="cuda", generator=g)).to(T[dt])
    d0 = padded((t, h), T[ht], 0, torch.randn((t, h), device="cuda", generator=g)) if with_dh else (None, None)
    want, wdw, e, edw = R.norm_backward(dys, hh, rstd, w, d0[0])
    dh = d0 if in_place else padded((t, h), T[ht])
    dxs = [(d, None) for d in dys[:copies]] if in_place else [padded((t, h), T[dt]) for _ in range(copies)]
    dw = padded((h,), torch.float32)
    print(f"[case] stream normbwd p={p} t={t} h={h} {dt} {ht} copies={copies} {in_place}", flush=True)
    B.ra_allreduce_rmsnorm_backward(dys, hh, rstd, w, dh[0], dh_in=d0[0], dxs=[d[0] for d in dxs], dweight=dw[0])
    R.check(dh[0], want, R.rounded(want, e, T[ht]), "dh")
    untouched(dh[1], 0, t * h)
    R.check(dw[0], wdw, R.rounded(wdw, edw, torch.float32), "dweight")
    untouched(dw[1], 0, h)
    for k, (d, flat) in enumerate(dxs):
        if k == 0:
            R.check(d, want, R.rounded(want, e, T[dt]), "dx")
        assert torch.equal(d, dxs[0][0])
        if flat is not None:
            untouched(flat, 0, t * h)


@pytest.mark.parametrize("p,t,v,h,dt,n_out", [
    (8, 8201, 1003, 4096, "bf16", 8), (8, 65539, 32000, 512, "f16", 8), (3, 33001, 5003, 2056, "f32", 3),
    (9, 131077, 91, 264, "bf16", 9), (1, 17001, 64, 16384, "f16", 1),
])
def test_embedding(p, t, v, h, dt, n_out):
    require_gpu()
    assert t * h * SIZE[dt] * n_out > STREAMS
    g = torch.Generator(device="cuda").manual_seed(t)
    table = torch.randn((v, h), device="cuda", generator=g).to(T[dt])
    ids = torch.randint(-3, v + 3, (t,), device="cuda", generator=g)
    b = B.ra_chunk_bounds(v, p)
    outs = [padded((t, h), T[dt]) for _ in range(n_out)]
    print(f"[case] stream embed p={p} t={t} v={v} h={h} {dt} n_out={n_out}", flush=True)
    B.ra_embedding([table[b[r]:b[r + 1]] for r in range(p)], ids, [o[0] for o in outs], scale=math.sqrt(h))
    want, err = R.embedding(table, ids, math.sqrt(h))
    R.check(outs[0][0], want, R.rounded(want, err, T[dt]), "y")
    for o, flat in outs:
        untouched(flat, 0, t * h)
        assert torch.equal(o.view(torch.uint8), outs[0][0].view(torch.uint8))
