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


def test_workspaces_elsewhere(monkeypatch):
    """A workspace that is not on the inputs' device, or that has gaps, is refused by every call (CPU
    stands for the inputs' device here, and the check of it is taken out of the way)."""
    from chunkwise_recurrent_prefill_gb300 import gla, hda, norm
    launched = []
    monkeypatch.setattr(hda, "_check_inputs", lambda q, *a: q.device)
    monkeypatch.setattr(norm, "_affine", lambda *a: None)
    for mod in (hda, norm):
        monkeypatch.setattr(mod, "_launch", lambda *a: launched.append(a) or 0)
    q = torch.zeros(1, 4, 2, 16)
    d, do = torch.zeros(2), torch.zeros(1, 4, 2, 16)
    calls = (lambda w: pkg.hda_fwd(q, q, q, d, 1.0, workspace=w),
             lambda w: pkg.hda_bwd(do, q, q, q, d, 1.0, workspace=w),
             lambda w: pkg.group_norm_fwd(do, 2, workspace=w))
    for call in calls:
        call(torch.zeros(64))
        n = len(launched)
        for bad in (torch.empty(64, device="meta"), torch.zeros(64)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)
        with pytest.raises(TypeError, match="workspace"):
            call(1 << 20)
        assert len(launched) == n
    with pytest.raises(ValueError, match="workspace"):
        gla._workspace(torch.zeros(64)[::2], torch.device("cpu"))


@pytest.mark.gpu
def test_workspaces_on_the_host():
    q = torch.zeros(1, 64, 2, 64, device="cuda")
    d, g = torch.zeros(2, device="cuda"), torch.zeros(1, 64, 2, 64, device="cuda")
    for bad in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, device="cuda")[::2]):
        for call in (lambda: pkg.hda_fwd(q, q, q, d, 1.0, workspace=bad),
                     lambda: pkg.hda_bwd(q, q, q, q, d, 1.0, workspace=bad),
                     lambda: pkg.gla_fwd(q, q, q, g, 1.0, workspace=bad)):
            with pytest.raises(ValueError, match="workspace"):
                call()
