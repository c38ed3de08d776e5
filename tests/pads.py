"""Device tensors with memory around them that a call has to leave alone."""

import math

import torch

from ring_all_reduce_schedule_amd import binding as B

PAD = 24          # elements behind a tensor


def padded(shape, dtype, off=0, fill=None):
    """A contiguous tensor `off` elements into its memory, with PAD elements behind it."""
    n = math.prod(shape)
    flat = torch.full((off + n + PAD,), 7.0, dtype=torch.float32, device="cuda").to(dtype)
    t = flat[off:off + n].view(shape)
    if fill is not None:
        t.copy_(fill)
    t.around = (flat, off)
    return t


def untouched(t):
    flat, off = t.around
    n = t.numel()
    ends = torch.cat([flat[:off].float(), flat[off + n:].float()])
    assert bool((ends == 7.0).all()), "elements outside the array were written"


def cut(x, p, off=0):
    """The ranks' pieces of x [tokens, vocab], each an array of its own."""
    b = B.ra_chunk_bounds(x.shape[1], p)
    return [padded((x.shape[0], b[r + 1] - b[r]), x.dtype, off, x[:, b[r]:b[r + 1]]) for r in range(p)]
