"""The optimizer binding's checks that need no GPU."""
import types

import pytest
import torch

from selective_state_space_05_gb300 import optim

HOST = types.SimpleNamespace(index=torch.Tensor.get_device(torch.zeros(1)))


def test_scales_must_be_dense():
    """A kernel reads one scale after another from the first's address."""
    blocks = [3]
    good = torch.arange(3.0)
    assert list(optim._scales([good], "s", HOST, blocks)) == [good.data_ptr()]
    wide = torch.zeros(3, 2)
    for bad in (wide[:, 0], torch.zeros(1).expand(3)):
        with pytest.raises(ValueError, match="dense"):
            optim._scales([bad], "s", HOST, blocks)
    with pytest.raises(ValueError, match="number or sizes"):
        optim._scales([torch.zeros(4)], "s", HOST, blocks)
    with pytest.raises(ValueError, match="required"):
        optim._scales(None, "s", HOST, blocks)


def test_shapes_and_not_only_sizes_must_match():
    want = [torch.Size([8, 4])]

    def table(t):
        return optim._table([t], "grads", torch.float32, HOST, want, optim._shape_of)
    good = torch.zeros(8, 4)
    assert list(table(good)[0]) == [good.data_ptr()]
    for bad in (torch.zeros(4, 8), torch.zeros(32), torch.zeros(8, 4, 1)):
        with pytest.raises(ValueError, match="grads: the tensors' number or sizes"):
            table(bad)
