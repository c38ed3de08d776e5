"""ra_grad_norm, ra_grad_clip and ra_allreduce_clip against their 64-bit forms (tests/answers_ref.py)."""

import math

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import answers_ref as A
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.pads import padded, untouched

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gradients(sizes, types, seed, off=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dtype = T[types[i % len(types)]]
        x = (sigma * 2.0 ** (i % 5 - 2) * torch.randn(n, device="cuda", generator=g)).to(dtype)
        out.append(padded((n,), dtype, off, x))
    return out


LISTS = [
    # sizes, types
    ([1], ["f32"]), ([7], ["bf16"]), ([8], ["f16"]), ([0, 5, 0], ["f32"]), ([2048], ["bf16"]), ([8191, 8192, 8193], ["f32", "bf16", "f16"]),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11], ["bf16", "f32", "f16"]), ([100_003, 1, 16_385], ["bf16"]), ([1 << 20, 3, 1 << 18], ["f32"]),
    ([17] * 127 + [1000], ["f16", "f32"]), ([64] * 128, ["f32"]), ([33] * 129, ["bf16"]), ([5000 + i for i in range(300)], ["bf16", "f32", "f16"]),
    ([(1 << 24) + 5], ["bf16"]), ([40_000_003], ["f16"]), ([1 << 22] * 20, ["bf16"]), ([11] * 2500, ["f32", "bf16"]),
]


@pytest.mark.parametrize("sizes,types", LISTS)
@pytest.mark.parametrize("off", [0, 1])
def test_norm(sizes, types, off):
    require_gpu()
    g = gradients(sizes, types, len(sizes), off)
    norm = padded((1,), torch.float32, 1)
    want, err = A.norm(g, 0.3)
    print(f"[case] norm of {len(sizes)} tensors, {sum(sizes)} elements", flush=True)
    B.ra_grad_norm(g, norm, scale=0.3)
    assert abs(float(norm.double()) - want) <= err
    untouched(norm)
    again = torch.empty(1, device="cuda")
    B.ra_grad_norm(B.TensorList(g), again, scale=0.3)
    assert torch.equal(again, norm)


@pytest.mark.parametrize("sizes,types", LISTS)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("how", ["in place", "outs", "wide", "half counted"])
@pytest.mark.parametrize("part", [0.5, 2.0])
def test_clip(sizes, types, off, how, part):
    require_gpu()
    g = gradients(sizes, types, len(sizes) + 1, off)
    counted = len(g) // 2 if how == "half counted" else None
    n, err = A.norm(g[:counted], 0.3)
    max_norm = max(part * n, 0.25)
    c, ec = A.factor(n, max_norm, 0.3)
    ec += c * (2.0 ** -39 + 2.0 ** -50)
    want = [A.scaled(t, c, ec, torch.float32 if how == "wide" else t.dtype) for t in g]
    norm = padded((1,), torch.float32, 1)
    outs = None
    if how in ("outs", "wide"):
        outs = [padded(t.shape, torch.float32 if how == "wide" else t.dtype, 3 if off else 0) for t in g]
    keep = [t.clone() for t in g]
    print(f"[case] clip of {len(sizes)} tensors, {sum(sizes)} elements, {how}", flush=True)
    B.ra_grad_clip(g, max_norm, norm, outs=outs, counted=counted, scale=0.3)
    torch.cuda.synchronize()
    assert abs(float(norm.double()) - n) <= err
    for got, (w, tol) in zip(outs or g, want):
        R.check(got, w, tol, "clipped")
        untouched(got)
    if outs:
        assert all(torch.equal(a, b) for a, b in zip(g, keep))
    untouched(norm)


@pytest.mark.parametrize("types,off", [(["bf16"], 0), (["bf16", "f16"], 1), (["f32"], 1)])
@pytest.mark.parametrize("how", ["in place", "outs", "wide"])
def test_lists_larger_than_the_caches(types, off, how):
    """More than 512 MiB, whose accesses go past the caches."""
    test_clip([(1 << 27) + 3, 5, 1 << 20, (1 << 27) + 9, 2], types, off, how, 0.5)


def test_a_factor_of_one_changes_no_bit():
    require_gpu()
    g = gradients([1000, 5, 8192 * 3 + 1], ["bf16", "f32", "f16"], 5)
    g[1][2] = -0.0
    keep = [t.clone() for t in g]
    norm = torch.empty(1, device="cuda")
    for max_norm in (1e9, math.inf):
        B.ra_grad_clip(g, max_norm, norm)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(g, keep))
    outs = [torch.empty_like(t) for t in g]
    B.ra_grad_clip(g, math.inf, norm, outs=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, keep))


@pytest.mark.parametrize("dt,size", [("f32", 3e38), ("bf16", 3e38), ("f16", 60000.0), ("f32", 1e-30), ("bf16", 1e-38), ("f16", 6e-8)])
def test_gradients_of_any_size(dt, size):
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = ((torch.rand(1000, device="cuda", generator=g, dtype=torch.float64) * 2 - 1) * size).to(T[dt])
    n, err = A.norm([x], 0.01)
    norm = torch.empty(1, device="cuda")
    B.ra_grad_norm([x], norm, scale=0.01)
    # below float32's smallest normal number, half of the smallest there is
    assert abs(float(norm.double()) - n) <= err + 2.0 ** -150
    out = torch.empty(1000, device="cuda")
    c, ec = A.factor(n, 0.5, 0.01)
    B.ra_grad_clip([x], 0.5, norm, outs=[out], scale=0.01)
    w, tol = A.scaled(x, c, ec, torch.float32)
    R.check(out, w, tol, "clipped")


def test_a_norm_beyond_float32():
    """It is infinite in float32; the factor, which comes from it in float64, is not zero."""
    require_gpu()
    x = torch.full((1000,), 2e38, device="cuda")
    norm, out = torch.empty(1, device="cuda"), torch.empty(1000, device="cuda")
    n = 2e38 * math.sqrt(1000)
    B.ra_grad_clip([x], 10.0, norm, outs=[out])
    assert norm.item() == math.inf
    w, tol = A.scaled(x, 10.0 / n, 10.0 / n * 2.0 ** -20, torch.float32)
    R.check(out, w, tol, "clipped")


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite(bad):
    require_gpu()
    x, y = torch.ones(5000, device="cuda"), torch.ones(300, device="cuda", dtype=torch.bfloat16)
    x[4321] = bad
    norm = torch.empty(1, device="cuda")
    B.ra_grad_norm([x, y], norm)
    assert norm.isnan().item() if math.isnan(bad) else norm.item() == math.inf
    B.ra_grad_clip([x, y], 1.0, norm)
    assert norm.isnan().item() if math.isnan(bad) else norm.item() == math.inf
    assert x[4321].isnan() and (y.isnan().all() if math.isnan(bad) else (y == 0).all())


def test_no_tensors():
    require_gpu()
    norm = torch.full((1,), 7.0, device="cuda")
    B.ra_grad_norm([], norm)
    assert norm.item() == 0.0
    norm.fill_(7.0)
    B.ra_grad_clip([torch.empty(0, device="cuda")], 1.0, norm)
    assert norm.item() == 0.0
    norm.fill_(7.0)
    B.ra_allreduce_clip([torch.empty(0, device="cuda")] * 1, 1.0, norm)
    assert norm.item() == 0.0
    x = torch.ones(10, device="cuda")
    B.ra_grad_clip([x], 1.0, norm, counted=0, scale=0.5)      # a norm of none: 0, and only scaled
    assert norm.item() == 0.0 and (x == 0.5).all()


FOLDS = [
    # p, n, dtype, offset
    (1, 1, "f32", 0), (2, 7, "bf16", 0), (3, 8, "f16", 0), (8, 2047, "bf16", 0), (8, 2048, "f32", 0), (9, 2049, "f16", 1),
    (64, 5003, "bf16", 0), (9, 1_000_003, "bf16", 0), (4, 1 << 20, "f32", 0), (8, (1 << 22) + 8, "bf16", 0), (5, 3_000_001, "f32", 3),
    (16, 1 << 19, "f16", 0), (2, 1 << 26, "bf16", 0), (1, 40_000_000, "f16", 0), (2, (1 << 27) + 2048 * 5 + 1, "bf16", 0), (2, 1 << 27, "f32", 0),
]


@pytest.mark.parametrize("p,n,dt,off", FOLDS)
@pytest.mark.parametrize("how", ["in place", "outs", "one out", "sum"])
def test_allreduce_clip(p, n, dt, off, how):
    require_gpu()
    dtype = T[dt]
    g = torch.Generator(device="cuda").manual_seed(n + p)
    bufs = [padded((n,), dtype, off, torch.randn(n, device="cuda", generator=g).to(dtype)) for _ in range(p)]
    mean = how != "sum"
    total, a = torch.zeros(n, dtype=R.F64, device="cuda"), torch.zeros(n, dtype=R.F64, device="cuda")
    for b in bufs:
        total += b.to(R.F64)
        a += b.to(R.F64).abs()
    eg = (p + 1) * R.U * a
    if mean:
        total, eg = total / p, eg / p + R.U * total.abs() / p
    op = "avg" if mean else "sum"
    keep = [b.clone() for b in bufs]
    # not clipped and not scaled, it is the sum rounded once
    plain, norm = [torch.empty_like(bufs[0])], padded((1,), torch.float32, 1)
    print(f"[case] allreduce clip p={p} n={n} {dt} {how}", flush=True)
    B.ra_allreduce_clip(bufs, math.inf, norm, plain, op=op)
    R.check(plain[0], total, R.rounded(total, eg, dtype), "sum")
    assert all(torch.equal(b, k) for b, k in zip(bufs, keep))
    del total, a, eg
    w, err = A.norm(plain, 1.0)
    assert abs(float(norm.double()) - w) <= err
    w, err = A.norm(plain, 0.5)
    c, ec = A.factor(w, 0.3 * w, 0.5)
    want, tol = A.scaled(plain[0], c, ec + c * 2.0 ** -39, dtype)
    outs = None
    if how in ("outs", "one out"):
        outs = [padded((n,), dtype, off) for _ in range(p if how == "outs" else 1)]
    B.ra_allreduce_clip(bufs, 0.3 * w, norm, outs, op=op, scale=0.5)
    torch.cuda.synchronize()
    assert abs(float(norm.double()) - w) <= err
    for o in outs or bufs:
        R.check(o, want, tol, "clipped")
        assert torch.equal(o, (outs or bufs)[0])
        untouched(o)
    if outs:
        assert all(torch.equal(b, k) for b, k in zip(bufs, keep))
    untouched(norm)


def test_outputs_in_the_place_of_other_ranks_buffers():
    require_gpu()
    bufs = [torch.full((5000,), float(r + 1), device="cuda") for r in range(4)]
    norm = torch.empty(1, device="cuda")
    other = torch.empty(5000, device="cuda")
    B.ra_allreduce_clip(bufs, math.inf, norm, [bufs[2], other, bufs[0]], op="sum")
    for t in (bufs[2], other, bufs[0]):
        assert (t == 10.0).all()
    assert (bufs[1] == 2.0).all() and (bufs[3] == 4.0).all()
