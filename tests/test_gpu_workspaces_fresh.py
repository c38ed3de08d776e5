"""The flag-driven ring on counters that its own call allocates, on an idle stream with nothing
queued in front of the kernel that polls them: the clear of the counters has to be ordered before
that kernel by the library."""

import pytest
import torch

import oracle
from ring_all_reduce_schedule_amd import binding as B
from ring_all_reduce_schedule_amd import inputs
from tests.gpu_util import first_diff, from_dev, require_gpu, same_bits, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,n,dtype", [(8, 300_007, "bfloat16"), (2, 4099, "float32"), (9, 1_000_003, "float16")])
def test_counters_allocated_by_the_call_on_an_idle_stream(p, n, dtype):
    require_gpu()
    xs = inputs.make_inputs(p, n, dtype, seed=21)
    src = to_dev(xs, dtype)
    bufs = [torch.empty_like(s) for s in src]
    want = oracle.ring_fold(xs, dtype)
    print(f"[case] fresh counters p={p} n={n} {dtype}", flush=True)
    s = torch.cuda.Stream()
    for k in range(6):
        for b, x in zip(bufs, src):
            b.copy_(x)
        torch.cuda.synchronize()
        B.ra_allreduce_ex(bufs, algo="ring_pipelined_flags", flags=B.RA_FLAG_RENEW_COUNTERS, stream=s)
        B.ra_stream_status(stream=s)
        for r, got in enumerate(from_dev(bufs, dtype)):
            assert same_bits(got, want, dtype), f"call {k} rank {r} at {first_diff(got, want, dtype)}"
