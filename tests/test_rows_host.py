"""Host side of the row operators: empty batches, the largest ones.  No call here reaches a kernel."""

import subprocess
import sys

import pytest

from ring_all_reduce_schedule_amd import binding as B
from tests.conftest import ROOT
from tests.test_rows_cpu import EMB_BWD, XENT, call


def in_child(code):
    """Runs `code` in a process of its own, which a fault of the library ends."""
    head = "from ring_all_reduce_schedule_amd import binding as B\n"
    return subprocess.run([sys.executable, "-c", head + code], cwd=ROOT, capture_output=True, text=True, timeout=120)


@pytest.mark.parametrize("vocab,p", [(1, 1), (4096, 2), (8192, 1), (32768, 2), (128000, 8), (1 << 24, 64)])
def test_cross_entropy_workspace_of_an_empty_batch(vocab, p):
    """Few tokens of a large vocabulary share their rows among workgroups: none are as many as 1024 / 0."""
    res = in_child(f"assert B.ra_cross_entropy_workspace(0, {vocab}, {p}) == 0")
    assert res.returncode == 0, (res.returncode, res.stderr)


def test_cross_entropy_of_an_empty_batch_has_empty_outputs():
    """An empty tensor's address is NULL: with no rows, that is no missing array."""
    assert call("ra_cross_entropy", XENT, tokens=0, loss=None, lse=None, grads=None, targets=None) == B.RA_OK
    assert call("ra_cross_entropy", XENT, tokens=0, loss=None, lse=None, grads=None, vocab=0) == B.RA_ERR_INVALID_ARG


def embedding_backward_takes(tokens, vocab, hidden):
    """The limits that include/ra.h states."""
    return tokens < 2 ** 31 - 4096 and -(-tokens // 16) * -(-hidden // 512) + -(-vocab // 8) <= 2 ** 24 - 1


@pytest.mark.parametrize("tokens,vocab,hidden", [
    (0, 1, 1), (1 << 27, 131072, 512), (268_000_000, 8, 512), (1 << 28, 8, 512), (234_881_008, 1 << 24, 512),
    (234_881_024, 1 << 24, 512), (16_000_000, 131072, 8192), (16_777_200, 8, 8192), (16_777_216, 8, 8192),
    ((1 << 31) - 4097, 1, 1), (1 << 31, 1, 1), (1 << 55, 8, 1), (1 << 58, 8, 1), (1 << 40, 1 << 24, 1 << 18),
])
def test_sizes_that_one_embedding_gradient_takes(tokens, vocab, hidden):
    """The workspace call and the call itself answer alike."""
    size = B.ctypes.c_int64(-1)
    rc = B.lib().ra_embedding_backward_workspace(tokens, vocab, hidden, B.ctypes.byref(size))
    # no workspace: a size that is taken is refused for that, unless there is nothing to sort
    back = call("ra_embedding_backward", EMB_BWD, tokens=tokens, vocab=vocab, hidden=hidden, ws=None, ws_bytes=0,
                accumulate=1)
    if embedding_backward_takes(tokens, vocab, hidden):
        assert rc == B.RA_OK and size.value >= 8 * tokens
        assert back == (B.RA_ERR_INVALID_ARG if tokens else B.RA_OK)
    else:
        assert rc == back == B.RA_ERR_UNSUPPORTED
