"""The eps of the norms may be anything that is a number, at the value that it has at the call (CPU tensors: shapes alone)."""
import pytest
import torch

from chunkwise_recurrent_prefill_gb300 import norm, qk_norm


def group(eps):
    return norm._shape(torch.zeros(3, 16), 2, eps, "none", None).eps


def heads(eps):
    q = torch.zeros(2, 5, 4, 16)
    return qk_norm._shape(q, q, "rms", "halves", eps, None).eps


@pytest.mark.parametrize("shape", [group, heads])
def test_an_eps_that_changes_in_place(shape):
    eps = torch.tensor(1e-6)
    first = shape(eps)
    assert abs(first - 1e-6) < 1e-12
    eps.fill_(1e-2)
    assert abs(shape(eps) - 1e-2) < 1e-8


@pytest.mark.parametrize("shape", [group, heads])
def test_an_eps_that_is_no_number(shape):
    assert shape(0) == 0 and shape(1e-5) > 0
    for bad in ("1e-6", None, [1e-6]):
        with pytest.raises(TypeError):
            shape(bad)
