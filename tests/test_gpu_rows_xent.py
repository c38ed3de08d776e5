"""ra_cross_entropy and its backward against their 64-bit forms (tests/rows_ref.py)."""

import math

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.test_gpu_rows_norm import T, padded, untouched

pytestmark = pytest.mark.gpu


def cut(x, p, off=0):
    """The ranks' pieces of x [tokens, vocab], each an array of its own."""
    b = B.ra_chunk_bounds(x.shape[1], p)
    return [padded((x.shape[0], b[r + 1] - b[r]), x.dtype, off, x[:, b[r]:b[r + 1]]) for r in range(p)]


def make(t, v, dtype, seed, valid=None, itype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (3 * torch.randn((t, v), device="cuda", generator=g)).to(dtype)
    y = torch.randint(0, valid or v, (t,), device="cuda", generator=g).to(itype)
    y[torch.rand(t, device="cuda", generator=g) < 0.2] = -100
    return x, y, g


CASES = [
    # p, tokens, vocab, valid, dtype, offset
    (1, 1, 1, 1, "f32", 0), (2, 3, 1, 1, "bf16", 0), (4, 5, 3, 2, "f16", 0), (3, 7, 20, 20, "bf16", 0),
    (1, 2, 511, 511, "f32", 0), (1, 5, 512, 512, "bf16", 0), (1, 5, 513, 500, "f16", 0), (2, 600, 1024, 1000, "bf16", 0),
    (8, 513, 4096, 4096, "bf16", 0), (8, 520, 4100, 4099, "bf16", 0), (9, 530, 5003, 5003, "f16", 1),
    (64, 515, 2000, 1999, "f32", 0), (64, 3, 32000, 32000, "bf16", 0), (8, 1, 128000, 128000, "bf16", 0),
    (8, 4, 128000, 128000, "f16", 0), (9, 2, 50017, 50001, "f32", 0), (8, 65, 32768, 32768, "bf16", 0),
    (8, 512, 16384, 16384, "bf16", 0), (8, 512, 16384, 16380, "f32", 3), (4, 514, 32768, 32768, "f16", 0),
    (4, 514, 33000, 33000, "f32", 0), (8, 512, 65536, 65536, "bf16", 0), (3, 513, 70001, 70000, "bf16", 0),
    (8, 96, 40000, 39990, "bf16", 0), (8, 97, 40000, 39990, "f16", 0), (3, 130, 70001, 70000, "bf16", 0),
    (5, 40, 66001, 66001, "f32", 1), (8, 300, 128000, 128000, "bf16", 0), (2, 61, 16390, 16390, "f16", 0),
    (3, 4, 1_000_003, 1_000_000, "bf16", 0), (3, 97, 1_000_003, 1_000_003, "f16", 0), (2, 3, 1 << 24, 1 << 24, "bf16", 0),
    (7, 98, 1 << 20, 1 << 20, "f32", 0), (8, 512, 131072, 131072, "bf16", 0), (1, 512, 151_937, 151_900, "f16", 0), (2, 512, 140_000, 140_000, "f32", 0),
]


@pytest.mark.parametrize("p,t,v,valid,dt,off", CASES)
@pytest.mark.parametrize("mode", ["loss", "grad", "in place"])
def test_cross_entropy(p, t, v, valid, dt, off, mode):
    require_gpu()
    dtype = T[dt]
    x, y, g = make(t, v, dtype, seed=t + v, valid=valid, itype=torch.int32 if t % 2 else torch.int64)
    if t > 4:
        x[1, : valid // 2] = -math.inf            # masked columns
        x[2, 1:valid] = torch.finfo(dtype).min    # masked with the type's lowest value
        x[3, :valid] = torch.finfo(dtype).min     # all of them
        x[4, :valid] = -math.inf                  # nothing left
        y[3], y[4] = valid - 1, 0
    if valid < v:
        x[:, valid:] = math.nan                   # padding is not read
    if t > 8:
        y[5], x[6, 0], y[6] = -1, math.nan, -5    # no loss: zeros, whatever the row holds
        y[7] = valid                              # no such column
    logits = cut(x, p, off)
    loss, lse = padded((t,), torch.float32), padded((t,), torch.float32)
    w = torch.rand(t, device="cuda", generator=g) if t % 3 else None
    grads = None if mode == "loss" else logits if mode == "in place" else cut(torch.zeros_like(x), p, off)
    print(f"[case] xent p={p} t={t} v={v} valid={valid} {dt} off={off} {mode}", flush=True)
    B.ra_cross_entropy([c[0] for c in logits], y, loss[0], lse[0], grads=grads and [c[0] for c in grads],
                       dloss=w, grad_scale=0.125, valid=valid)
    wl, wz, wg, el, ez, eg = R.xent(x, y.long(), valid, w, 0.125)
    keep = torch.ones(t, dtype=torch.bool, device="cuda")
    if t > 8:
        keep[6] = False                           # NaN: its lse is NaN too
        assert loss[0][6] == 0 and bool(lse[0][6].isnan())
    R.check(loss[0][keep], wl[keep], el[keep] + R.U * wl[keep].abs().nan_to_num(), "loss")
    R.check(lse[0][keep], wz[keep], ez[keep], "lse")
    untouched(loss[1], 0, t)
    untouched(lse[1], 0, t)
    if grads is not None:
        got = torch.cat([c[0] for c in grads], 1)
        wg = torch.where(keep.unsqueeze(1), wg, 0.0)
        R.check(got, wg, R.rounded(wg, torch.where(keep.unsqueeze(1), eg, 0.0), dtype), "grad")
        for c, flat in grads:
            untouched(flat, off, c.numel())
    if mode != "in place":
        assert torch.equal(torch.cat([c[0] for c in logits], 1).nan_to_num(), x.nan_to_num())


@pytest.mark.parametrize("p,t,v,valid,dt,off", [c for c in CASES if c[1] < 515 or c[2] < 6000])
def test_backward_from_lse(p, t, v, valid, dt, off):
    require_gpu()
    dtype = T[dt]
    x, y, g = make(t, v, dtype, seed=2 * t + v, valid=valid)
    if t > 4:
        x[1, : valid // 2] = -math.inf
        x[4, :valid] = -math.inf
        y[4] = 0
    logits = cut(x, p, off)
    lse = torch.empty(t, device="cuda")
    B.ra_cross_entropy([c[0] for c in logits], y, lse=lse, valid=valid)
    w = torch.rand(t, device="cuda", generator=g)
    grads = cut(torch.zeros_like(x), p, off)
    print(f"[case] xentbwd p={p} t={t} v={v} valid={valid} {dt} off={off}", flush=True)
    B.ra_cross_entropy_backward([c[0] for c in logits], y, lse, [c[0] for c in grads], dloss=w, valid=valid)
    _, wz, wg, _, ez, eg = R.xent(x, y, valid, w, 1.0)
    # the given lse is off by ez, which is ez relative in exp(x - lse); the difference x - lse
    # in float32 by u of itself at most |lse| + |x|
    more = (ez + R.U * wz.abs().nan_to_num(posinf=0, neginf=0)).unsqueeze(1) + \
        R.U * x.double().abs().nan_to_num(nan=0, posinf=0, neginf=0)
    more = more * (wg.abs() + w.double().unsqueeze(1) * torch.exp(x.double() - wz.unsqueeze(1)).nan_to_num(0, 0, 0))
    got = torch.cat([c[0] for c in grads], 1)
    R.check(got, wg, R.rounded(wg, eg + more.nan_to_num(0, 0, 0), dtype), "grad")
    for c, flat in grads:
        untouched(flat, off, c.numel())
    B.ra_cross_entropy_backward([c[0] for c in logits], y, lse, [c[0] for c in logits], dloss=w, valid=valid)
    for a, b in zip(logits, grads):
        assert torch.equal(a[0], b[0])


def test_plus_infinity_and_nan_poison_their_token_only():
    require_gpu()
    for t, v in ((4, 40), (4, 20000), (600, 9000)):
        x, _, _ = make(t, v, torch.float32, seed=v)
        y = torch.full((t,), v - 1, device="cuda")
        x[0, 3], x[1, v // 2] = math.inf, math.nan
        logits = [c[0] for c in cut(x, 3)]
        loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        B.ra_cross_entropy(logits, y, loss, lse, grads=logits)
        got = torch.cat(logits, 1)
        assert bool(loss[:2].isnan().all()) and bool(got[:2].isnan().all())
        assert bool(loss[2:].isfinite().all()) and bool(got[2:].isfinite().all())


@pytest.mark.parametrize("t,v", [(3, 40000), (130, 40000), (130, 700), (3, 5)])
@pytest.mark.parametrize("size", [1e-30, 1e4, 1e8, 3e9, 1e12, 1e37, 3e38])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logits_of_any_size(t, v, size, dt):
    """Far beyond where 2^(x log2 e - c) is a float32 number, and with ties at the top."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(v + t)
    x = ((2 * torch.rand((t, v), device="cuda", generator=g) - 1) * size).to(T[dt])
    x[0, -1] = x[0, 0] = x[0].max()
    y = torch.randint(0, v, (t,), device="cuda", generator=g)
    y[0] = v - 1
    grads = [c[0] for c in cut(torch.zeros_like(x), 3 if v > 5 else 2)]
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    print(f"[case] xent size={size} t={t} v={v} {dt}", flush=True)
    B.ra_cross_entropy([c[0] for c in cut(x, len(grads))], y, loss, lse, grads=grads)
    wl, wz, wg, el, ez, eg = R.xent(x, y, v, None, 1.0)
    big = torch.finfo(torch.float32).max
    wl = torch.where(wl > big * (1 + 2.0 ** -25), math.inf, wl)       # a difference float32 does not hold
    R.check(loss, wl, el + R.U * wl.abs(), "loss")
    R.check(lse, wz, ez, "lse")
    R.check(torch.cat(grads, 1), wg, R.rounded(wg, eg, T[dt]), "grad")


def test_gradient_against_differences():
    require_gpu()
    t, v = 6, 1003
    x, y, g = make(t, v, torch.float32, seed=5)
    grads = [c[0] for c in cut(torch.zeros_like(x), 4)]
    w = torch.rand(t, device="cuda", generator=g)
    B.ra_cross_entropy([c[0] for c in cut(x, 4)], y, grads=grads, dloss=w)
    got = torch.cat(grads, 1).double()

    def f(x):
        live = y >= 0
        at = y.clamp_min(0).unsqueeze(1)
        return (torch.where(live, torch.logsumexp(x, 1) - x.gather(1, at).squeeze(1), 0.0) * w.double()).sum()

    s = 1e-5
    for _ in range(4):
        d = torch.randn((t, v), device="cuda", generator=g).double()
        num = (f(x.double() + s * d) - f(x.double() - s * d)) / (2 * s)
        assert abs(float(num - (got * d).sum())) <= 1e-5 * float((got * d).abs().sum()) + 1e-9


def test_columns_past_two_to_the_32():
    """40,000 tokens of 131,072 columns: 5.2e9 logits."""
    require_gpu()
    t, v = 40_000, 131_072
    x = torch.zeros((t, v), dtype=torch.bfloat16, device="cuda")
    y = torch.arange(t, device="cuda") % v
    x[-1, 7] = 4.0
    loss = torch.empty(t, device="cuda")
    print("[case] xent 40000 x 131072", flush=True)
    B.ra_cross_entropy([x], y, loss, grads=[x])
    assert bool((loss[:-1] - math.log(v)).abs().max() < 1e-4)
    p = torch.tensor(1.0 / v).to(torch.bfloat16)
    assert bool((x[0, 1:] == p.item()).all()) and bool((x[-2, : t - 2] == p.item()).all())
    z = v - 1 + math.exp(4.0)
    assert abs(float(x[-1, 7]) - math.exp(4.0) / z) < 2 ** -8 * math.exp(4.0) / z
    assert abs(float(x[-1, t - 1]) - (1 / z - 1)) < 2 ** -8
