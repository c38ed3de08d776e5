"""Every unit of a row counts once in ra_token_logprobs: rows nearly all of whose probability lies in one
column, which is in turn in each unit of eight, and at the ends of each chunk, of each rank's piece and of
the valid columns.  (Among thousands of ordinary logits a unit that is left out or taken twice
changes the sums by less than what float32 may be off from them.)"""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import answers_ref as A
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.pads import cut

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEEP = 20.0        # how far the other logits lie below the one


def columns(p, v, valid):
    """A column of each unit, another place in it from unit to unit, and what stands at a border."""
    b = B.ra_chunk_bounds(v, p)
    at = set()
    for lo, hi in zip(b, b[1:]):
        at.update({lo, hi - 1} if hi > lo else ())
        at.update(lo + i + i // 8 % 8 for i in range(0, hi - lo, 8))
        for i in range(0, hi - lo, 512):
            at.update({lo + i, lo + i + 511, lo + i + 7, lo + i + 504})
    at.update({valid - 1, valid - 8, 0})
    return sorted(c for c in at if 0 <= c < valid)


def sums(base, scale):
    """Of e^y and e^y y over the row, and of e^y y^2, in 64 bits."""
    y = base.double() * scale
    e = y.exp()
    return e, y, e.sum(), (e * y).sum(), (e * y * y).sum()


CASES = [
    # p, tokens in a call, vocab, valid, dtype, offset, top
    (64, 100, 450, 449, "bf16", 0, 3),              # pieces shorter than a unit
    (1, 20, 9, 9, "f32", 0, 3), (3, 300, 3000, 3000, "bf16", 0, 3), (3, 300, 3001, 2500, "f16", 1, 3),
    (1, 300, 5000, 4990, "f32", 0, 64), (2, 300, 1024, 1000, "bf16", 0, 3),
    (8, 2100, 16384, 16384, "bf16", 0, 3), (7, 2100, 16385, 16380, "f32", 1, 20),
    (1, 150, 151_937, 151_900, "f16", 0, 20), (2, 700, 131_072, 131_072, "f32", 0, 3),
    (2, 2100, 131_072, 131_072, "bf16", 0, 20),     # past the caches
    # rows in parts
    (8, 4, 128_000, 128_000, "f16", 0, 20), (8, 16, 128_000, 127_999, "bf16", 0, 3), (9, 16, 50_017, 50_001, "f32", 1, 64),
    (64, 12, 40_000, 39_990, "bf16", 0, 3), (5, 330, 300_007, 300_000, "bf16", 1, 3), (3, 64, 1_000_003, 1_000_000, "f32", 0, 3),
]


@pytest.mark.parametrize("p,t,v,valid,dt,off,top", CASES)
def test_every_unit_counts_once(p, t, v, valid, dt, off, top):
    require_gpu()
    dtype, scale = T[dt], 1.0
    g = torch.Generator(device="cuda").manual_seed(v)
    base = (torch.randn(v, device="cuda", generator=g) - DEEP).to(dtype)
    base[valid:] = torch.nan                                     # padding is not read
    pieces = cut(base.expand(t, v), p, off)
    b = B.ra_chunk_bounds(v, p)
    # the ordinary columns' best, more than are asked for: one of them may be the row's one
    k = min(top, valid)
    others = A.best(base[:valid].unsqueeze(0), min(k + 1, valid)).squeeze(0)
    e, y, s0, s1, s2 = sums(base[:valid], scale)
    at = torch.tensor(columns(p, v, valid), device="cuda")
    piece = torch.bucketize(at, torch.tensor(b[1:], device="cuda"), right=True)
    print(f"[case] {len(at)} columns, p={p} t={t} v={v} {dt}", flush=True)
    f = dict(dtype=torch.float32, device="cuda")
    bad = torch.zeros(4, dtype=torch.bool, device="cuda")
    rows = torch.arange(t, device="cuda")
    depth = 4 * (256 + valid / 512 + 86)                         # as for answers_ref.logprobs
    for lo in range(0, len(at), t):
        which = (lo + rows) % len(at)                            # the last call's rows go round
        c, r = at[which], piece[which]
        for q in range(p):
            here = (r == q)
            pieces[q].copy_(torch.where((torch.arange(b[q], b[q + 1], device="cuda") == c.unsqueeze(1)) & here.unsqueeze(1),
                                        torch.zeros((), dtype=dtype, device="cuda"), base[b[q]:b[q + 1]]))
        lp, ent, lse = (torch.full((t,), 7.0, **f) for _ in range(3))
        ids, tlp = torch.full((t, k), -7, device="cuda"), torch.full((t, k), 7.0, **f)
        B.ra_token_logprobs(pieces, c, lp, ent, lse, ids, tlp, scale=scale, valid=valid)
        lp2, ent2, lse2 = (torch.full((t,), 7.0, **f) for _ in range(3))
        B.ra_token_logprobs(pieces, c, lp2, ent2, lse2, scale=scale, valid=valid)
        z = s0 - e[c] + 1.0
        mean = -(s1 - e[c] * y[c]) / z                           # of how far below the one
        squares = (s2 - e[c] * y[c] * y[c]) / z
        ln_z = z.log()
        ez = (depth + 20 + 4 * mean) * R.U
        eln = ez + 2.0 ** -22 + 4 * R.U * ln_z
        eent = eln + mean * (ez + depth * R.U + 10 * R.U) + 4 * R.U * squares + R.U * (ln_z + 2 * mean)
        near = eln + 3 * R.U * ln_z + 2.0 ** -140
        for a, a2, want, err, i in ((lp, lp2, -ln_z, near, 0), (ent, ent2, ln_z + mean, eent + R.U * (ln_z + mean), 1),
                                    (lse, lse2, ln_z, near, 2)):
            bad[i] |= ((a.double() - want).abs() > err).any() | (a != a2).any()
        # the one, then the others without it
        rest = others.expand(t, -1)
        keep = rest != c.unsqueeze(1)
        keep &= keep.cumsum(1) <= k - 1
        want = torch.cat([c.unsqueeze(1), rest[keep].view(t, -1)], 1) if k > 1 else c.unsqueeze(1)
        bad[3] |= (ids != want).any() | (tlp[:, 0] != lp).any()
    assert bad.tolist() == [False] * 4, dict(zip(("logprob", "entropy", "lse", "alternatives"), bad.tolist()))


@pytest.mark.parametrize("t,v,dt", [(3, 131072, "bf16"), (300, 131072, "bf16"), (300, 4096, "f32"), (300, 50017, "f16")])
def test_the_best_column_alone(t, v, dt):
    """One alternative, of rows whose best lie in few threads, with ties."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((t, v), device="cuda", generator=g)
    col = torch.arange(v, device="cuda")
    x += torch.where(col % 512 < 8, 100.0, 0.0)
    x[::2, ::512] = 200.0
    x[1] = 3.0                                                   # all equal
    x[2, :v // 2] = -torch.inf
    x = x.to(T[dt])
    for p in (1, 2, 8):
        one, lp = torch.full((t, 1), -7, device="cuda"), torch.full((t, 1), 7.0, device="cuda")
        print(f"[case] the best column p={p} t={t} v={v} {dt}", flush=True)
        B.ra_token_logprobs(cut(x, p), top_ids=one, top_logprobs=lp)
        assert torch.equal(one, A.best(x, 1))
        want, err = A.logprobs(x, one[:, 0], 1.0, v, 1)
        R.check(lp, want[4], R.rounded(want[4], err[4], torch.float32), "top_logprobs")
