"""ra_embedding and its backward against their 64-bit forms (tests/rows_ref.py)."""

import math

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.test_gpu_rows_norm import T, padded, untouched

pytestmark = pytest.mark.gpu


def cut(table, p, off=0):
    b = B.ra_chunk_bounds(table.shape[0], p)
    return [padded((b[r + 1] - b[r], table.shape[1]), table.dtype, off, table[b[r]:b[r + 1]]) for r in range(p)]


def ids_of(kind, t, v, g, itype=torch.int64):
    if kind == "same":
        ids = torch.full((t,), v // 2, device="cuda")
    elif kind == "zipf":
        ids = (torch.exp(torch.rand(t, device="cuda", generator=g).double() * math.log(v + 1)) - 1).long().clamp(0, v - 1)
    elif kind == "none":
        ids = torch.full((t,), -1, device="cuda")
    elif kind == "far":
        ids = torch.randint(-3, v + 3, (t,), device="cuda", generator=g)
    else:
        ids = torch.randint(0, v, (t,), device="cuda", generator=g)
    return ids.to(itype)


FORWARD = [
    (1, 1, 1, 1, "f32", 0), (2, 5, 1, 3, "bf16", 0), (9, 17, 5, 7, "f16", 0), (8, 16, 32000, 4096, "bf16", 0),
    (8, 300, 1000, 512, "bf16", 0), (8, 300, 1003, 513, "f16", 1), (64, 40, 100, 1001, "f32", 0),
    (3, 2, 50, 20008, "bf16", 0), (4, 1030, 77, 64, "f32", 0), (8, 129, 500, 2056, "bf16", 0),
]


@pytest.mark.parametrize("p,t,v,h,dt,off", FORWARD)
@pytest.mark.parametrize("kind", ["far", "zipf"])
def test_embedding(p, t, v, h, dt, off, kind):
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(t + v + h)
    table = torch.randn((v, h), device="cuda", generator=g).to(T[dt])
    ids = ids_of(kind, t, v, g, torch.int32 if t % 2 else torch.int64)
    for n_out in {1, p}:
        outs = [padded((t, h), T[dt], off) for _ in range(n_out)]
        print(f"[case] embed p={p} t={t} v={v} h={h} {dt} off={off} {kind} n_out={n_out}", flush=True)
        B.ra_embedding([c[0] for c in cut(table, p, off)], ids, [o[0] for o in outs], scale=math.sqrt(h))
        want, err = R.embedding(table, ids, math.sqrt(h))
        for o, flat in outs:
            R.check(o, want, R.rounded(want, err, T[dt]), "y")
            untouched(flat, off, t * h)


BACKWARD = [
    # p, tokens, vocab, hidden, dy's type, table's type, ids, offset
    (1, 1, 1, 1, "f32", "f32", "any", 0), (2, 3, 5, 3, "bf16", "bf16", "any", 0), (3, 16, 4, 8, "f16", "f32", "any", 0),
    (9, 17, 5, 9, "f16", "f16", "far", 0), (4, 33, 40, 64, "bf16", "f32", "same", 0), (8, 1003, 503, 101, "bf16", "bf16", "zipf", 0),
    (8, 100, 30, 2056, "bf16", "f32", "far", 0), (9, 1003, 5003, 1001, "f16", "f16", "zipf", 1), (2, 50, 9, 40, "f32", "f32", "none", 0),
    (64, 4096, 33, 24, "f32", "f32", "zipf", 0), (8, 4097, 300, 16, "bf16", "f32", "zipf", 0), (8, 5000, 70000, 8, "f16", "f32", "any", 0),
    (8, 20000, 600, 40, "bf16", "bf16", "zipf", 0), (5, 12345, 300_001, 9, "f32", "f32", "far", 0), (1, 9000, 2, 17, "bf16", "f32", "same", 0),
    (8, 70000, 131072, 16, "bf16", "f32", "zipf", 0), (3, 8192, 511, 8, "f32", "f32", "any", 0), (3, 8193, 512, 8, "f32", "f32", "far", 0),
    (9, 3, 70144, 192, "f32", "f32", "any", 0), (2, 21, 39548, 191, "f16", "f16", "far", 1), (4, 9, 300_000, 3, "bf16", "f32", "any", 0),
]


@pytest.mark.parametrize("p,t,v,h,dt,tt,kind,off", BACKWARD)
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward(p, t, v, h, dt, tt, kind, off, accumulate):
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(t + v + h)
    dy = padded((t, h), T[dt], off, torch.randn((t, h), device="cuda", generator=g))[0]
    ids = ids_of(kind, t, v, g, torch.int32 if t % 2 else torch.int64)
    old = torch.randn((v, h), device="cuda", generator=g).to(T[tt])
    tables = cut(old, p, off)
    print(f"[case] embedbwd p={p} t={t} v={v} h={h} {dt} {tt} {kind} off={off} acc={accumulate}", flush=True)
    B.ra_embedding_backward(dy, ids, [c[0] for c in tables], scale=1.5, accumulate=accumulate)
    want, err, has = R.embedding_backward(dy, ids, v, 1.5, old if accumulate else None)
    got = torch.cat([c[0] for c in tables])
    tol = R.rounded(want, err, T[tt])
    R.check(got, want, tol, "dtable")
    rest = ~has
    assert torch.equal(got[rest], old[rest] if accumulate else torch.zeros_like(old[rest]))
    for c, flat in tables:
        untouched(flat, off, c.numel())
    # the same bits again: the ids alone decide the order of the sums
    again = cut(old, p, off)
    B.ra_embedding_backward(dy, ids, [c[0] for c in again], scale=1.5, accumulate=accumulate)
    assert all(torch.equal(a[0], b[0]) for a, b in zip(tables, again))


def test_sums_follow_the_positions():
    """Terms that cancel only in their order: 2^24, 1, -2^24 in float32 gives 0 in the order
    given and 1 in others; every run lies inside one stretch of sixteen."""
    require_gpu()
    for t in (48, 4800):                    # both sorts
        ids = torch.arange(t, device="cuda") % (t // 3)
        vals = torch.tensor([2.0 ** 24, 1.0, -2.0 ** 24], device="cuda").repeat_interleave(t // 3)
        dy = vals.unsqueeze(1).repeat(1, 8).contiguous()
        d = torch.empty((t // 3, 8), device="cuda")
        B.ra_embedding_backward(dy, ids, [d])
        crosses = (torch.arange(t // 3, device="cuda") * 3 % 16) > 13
        assert bool((d[~crosses] == 0).all())


def test_no_tokens():
    require_gpu()
    d = torch.ones((5, 9), device="cuda")
    none, dy = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty((0, 9), device="cuda")
    B.ra_embedding_backward(dy, none, [d], accumulate=True)
    assert bool((d == 1).all())
    B.ra_embedding_backward(dy, none, [d])
    assert bool((d == 0).all())
    B.ra_embedding([d], none, [torch.empty((0, 9), device="cuda")])


def test_tables_past_two_to_the_32():
    """A table of 1,100,000 rows of 4096: 4.5e9 elements."""
    require_gpu()
    v, h = 1_100_000, 4096
    table = torch.zeros((v, h), dtype=torch.bfloat16, device="cuda")
    table[v - 1], table[v // 2] = 3.0, 5.0
    b = B.ra_chunk_bounds(v, 2)
    pieces = [table[b[r]:b[r + 1]] for r in range(2)]
    ids = torch.tensor([v - 1, 0, v // 2, v - 1], device="cuda")
    y = torch.empty((4, h), dtype=torch.bfloat16, device="cuda")
    print("[case] embed 1100000 x 4096", flush=True)
    B.ra_embedding(pieces, ids, [y])
    assert [float(r[-1]) for r in y] == [3.0, 0.0, 5.0, 3.0]
    B.ra_embedding_backward(y, ids, pieces)
    assert float(table[v - 1, 0]) == 6.0 and float(table[v // 2, h - 1]) == 5.0
    assert int((table != 0).any(1).sum()) == 2
