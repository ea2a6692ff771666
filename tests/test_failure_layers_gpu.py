"""Failure detection without a GPU fault, in the operators around a recurrent layer: a bounded wait that runs out.

With GLA_TEST_STALL_ONE_LOAD set when a process starts, its first call leaves out the load of one chunk (a barrier that
nothing completes). Every wait that depends on it gives up after its limit, the kernels raise the library's device error
word, let what they asked for land and return: the host reads GLA_ERR_DEVICE_TIMEOUT, and the next call is correct. The
library reads the variable once per process, so each call has a child process (tests/stall_layer_child.py).
"""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# A warp waits 2 s until it gives up, and as long for each of the two loads that may be on their way; a call has up to two
# kernels that load.
@pytest.mark.parametrize("call", ["scan", "scan in segments", "scan gradients", "norm", "norm gradients"])
def test_a_wait_that_runs_out(call):
    env = dict(os.environ, GLA_TEST_STALL_ONE_LOAD="1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "stall_layer_child.py"), call], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["status_before"] == 0 and out["status_cleared"] == 0 and out["status_after"] == 0, out
    assert out["status_stalled"] == 7, out            # GLA_ERR_DEVICE_TIMEOUT
    assert 1.0 < out["waited_s"] < 30.0, out
