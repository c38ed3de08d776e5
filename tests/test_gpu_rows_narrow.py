"""The embedding's gradient where a wave has few lanes left: rows of a few units, and rows whose
last wave has one.  A stretch's 16 keys and positions are loaded a lane to a key, by waves
whose lanes may have nothing else to do."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
from tests.gpu_util import require_gpu
from tests.test_gpu_rows_embed import cut, ids_of
from tests.test_gpu_rows_norm import T, padded, untouched

pytestmark = pytest.mark.gpu

PAIRS = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")]


@pytest.mark.parametrize("dt,tt", PAIRS)
@pytest.mark.parametrize("h", [1, 8, 9, 128, 136, 139, 520, 521, 2056])
def test_embedding_backward_of_narrow_rows(h, dt, tt):
    require_gpu()
    t, v, p = 333, 91, 3
    g = torch.Generator(device="cuda").manual_seed(h)
    dy = padded((t, h), T[dt], 0, torch.randn((t, h), device="cuda", generator=g))[0]
    ids = ids_of("zipf", t, v, g)
    ids[::50] = -1
    for accumulate in (False, True):
        old = torch.randn((v, h), device="cuda", generator=g).to(T[tt])
        tables = cut(old, p)
        print(f"[case] narrow embedbwd h={h} {dt} {tt} acc={accumulate}", flush=True)
        B.ra_embedding_backward(dy, ids, [x[0] for x in tables], scale=1.5, accumulate=accumulate)
        want, err, _ = R.embedding_backward(dy, ids, v, 1.5, old if accumulate else None)
        b = B.ra_chunk_bounds(v, p)
        for r, (x, flat) in enumerate(tables):
            w = want[b[r]:b[r + 1]]
            R.check(x, w, R.rounded(w, err[b[r]:b[r + 1]], T[tt]), "dtable")
            untouched(flat, 0, x.numel())
