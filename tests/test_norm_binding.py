"""Shapes and strides as the group norm's binding reads them (CPU tensors: refused before any
launch)."""
import pytest
import torch

from chunkwise_recurrent_prefill_gb300 import norm


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(2, 1, 16).expand(2, 9, 16),             # one position for all
    lambda: torch.zeros(2, 5, 1, 16).expand(2, 5, 7, 16),       # of the inner of two dimensions
    lambda: torch.zeros(2, 1, 7, 16).expand(2, 5, 7, 16),       # of the outer one
    lambda: torch.zeros(1, 9, 16).expand(2, 9, 16),             # one entry for all
    lambda: torch.zeros(2, 1, 1, 16).expand(2, 5, 7, 16),
])
def test_repeated_positions_are_refused(make):
    """A stride of zero is no spacing that a kernel can walk. (Taken for C, it read past the end.)"""
    t = make()
    x = torch.zeros(t.shape)
    for args in ((t, None), (x, t), (x, None, t)):
        with pytest.raises(ValueError, match="positive|evenly"):
            norm._shape(args[0], 4, 1e-5, "none", *args[1:])


def test_strides_of_views():
    x = torch.zeros(3, 5, 7, 48)
    sh = norm._shape(x[..., 16:32], 4, 1e-5, "none", None)
    assert (sh.N, sh.L, sh.C, sh.x_n, sh.x_l) == (3, 35, 16, 35 * 48, 48)
    sh = norm._shape(x[:, :, :1], 4, 1e-5, "none", x[:, :, 3:4])
    assert (sh.L, sh.x_l, sh.gate_n, sh.gate_l) == (5, 7 * 48, 35 * 48, 7 * 48)
    with pytest.raises(ValueError, match="evenly"):
        norm._shape(x[:, :, :2], 4, 1e-5, "none", None)
    # a dimension of one element may have any stride
    one = torch.zeros(1, 1, 16).expand(1, 1, 16)
    assert norm._shape(one, 4, 1e-5, "none", None).L == 1
    sh = norm._shape(torch.zeros(4, 1, 16).as_strided((4, 1, 16), (16, 0, 1)), 4, 1e-5, "none", None)
    assert (sh.x_n, sh.x_l) == (16, 16)


@pytest.mark.parametrize("groups", [2.5, 2.0, "2", None])
def test_groups_that_are_not_whole_numbers_are_refused(groups):
    norm._shape(torch.zeros(3, 16), 2, 1e-5, "none", None)     # (a shape that has been seen with 2)
    with pytest.raises(TypeError):
        norm._shape(torch.zeros(3, 16), groups, 1e-5, "none", None)
