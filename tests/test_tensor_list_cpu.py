"""A TensorList looks at every tensor's address and length before a call uses its table (host only)."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B


@pytest.fixture
def held(monkeypatch):
    """A TensorList of host tensors: the class wants device tensors, of which there are none here."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    return B.TensorList([torch.randn(5 + i) for i in range(7)] + [torch.empty(0), torch.randn(3, 4)])


def test_unchanged_tensors_pass(held):
    for t in held.tensors:
        t.normal_()
    held.tensors[8].resize_(4, 3)                     # the same elements
    assert B._marshalled(held) is held


@pytest.mark.parametrize("which", range(9))
@pytest.mark.parametrize("how", ["set_", "data", "grown", "shrunk", "storage"])
def test_each_tensor_is_looked_at(held, which, how):
    t = held.tensors[which]
    if t.numel() == 0 and how != "grown":
        pytest.skip("without elements it has no address, and nothing of it is read")
    if how == "set_":
        t.set_(torch.zeros(1000)[500:500 + t.numel()])
    elif how == "data":
        t.data = torch.zeros(t.numel() + 1)[1:]
    elif how == "grown":
        t.resize_(100_000)
    elif how == "shrunk":
        t.resize_(t.numel() - 1)
    else:
        t.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="re-pointed"):
        B._marshalled(held)
