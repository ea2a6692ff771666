"""Arguments that are not tensors, as the bindings of the decay attention and the state pages refuse
them (CPU tensors: nothing is launched)."""
import numpy as np
import pytest
import torch

import chunkwise_recurrent_prefill_gb300 as pkg
from chunkwise_recurrent_prefill_gb300 import build_ext


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_ext.build()


def test_attention():
    q = k = v = torch.zeros(1, 4, 2, 16)
    d, do = torch.zeros(2), torch.zeros(1, 4, 2, 16)
    for bad in (None, [0.0, 0.0], np.zeros(2, np.float32)):
        with pytest.raises(TypeError, match="decay must be a torch.Tensor"):
            pkg.hda_fwd(q, k, v, bad, 1.0)
        with pytest.raises(TypeError, match="decay must be a torch.Tensor"):
            pkg.hda_bwd(do, q, k, v, bad, 1.0)
        with pytest.raises(TypeError, match="do must be a torch.Tensor"):
            pkg.hda_bwd(bad, q, k, v, d, 1.0)
        with pytest.raises(TypeError, match="decay must be a torch.Tensor"):
            pkg.hda_step(q[:, 0], k[:, 0], v[:, 0], bad, 1.0, torch.zeros(1, 2, 16, 16))
        with pytest.raises(TypeError, match="decay must be a torch.Tensor"):
            pkg.hda_path_for(q, k, v, bad)


def test_step_states(monkeypatch):
    """(The check of the device comes before, so it is taken out of the way.)"""
    from chunkwise_recurrent_prefill_gb300 import hda
    monkeypatch.setattr(hda, "_check_inputs", lambda q, *a: q.device)
    q = torch.zeros(1, 2, 16)
    for bad in (None, 1.0, np.zeros((1, 2, 16, 16), np.float32)):
        with pytest.raises(TypeError, match="S must be a torch.Tensor"):
            pkg.hda_step(q, q, q, torch.zeros(2), 1.0, bad)
    with pytest.raises(ValueError, match="S: shape"):
        pkg.hda_step(q, q, q, torch.zeros(2), 1.0, torch.tensor(0.0))


def test_pages(monkeypatch):
    from chunkwise_recurrent_prefill_gb300 import pages
    monkeypatch.setattr(pages, "_pool", lambda pool: (4, 64))
    pool, table = torch.zeros(4, 16), torch.zeros(3, 1, dtype=torch.int32)
    free, count, one = (torch.zeros(n, dtype=torch.int32) for n in (4, 1, 1))
    with pytest.raises(TypeError, match="src must be"):
        pkg.pages_copy(pool, [0], one)
    with pytest.raises(TypeError, match="parents must be"):
        pkg.pages_fork(pool, table, free, count, [0], one)
    with pytest.raises(TypeError, match="table must be"):
        pkg.pages_compact(pool, [[0]], free, count)
    with pytest.raises(TypeError, match="table must be"):
        pkg.pages_free(None, free, count, one)
    with pytest.raises(TypeError, match="free must be"):
        pkg.pages_free(table, None, count, one)
    with pytest.raises(TypeError, match="table must be"):
        pkg.pages_workspace_size([[0]], free)
    with pytest.raises(TypeError, match="free must be"):
        pkg.pages_workspace_size(table, 4)
