"""Host side of the row operators: empty batches.  No call here reaches a kernel."""

import subprocess
import sys

import pytest

from ring_all_reduce_schedule_amd import binding as B
from tests.conftest import ROOT
from tests.test_rows_cpu import XENT, call


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
