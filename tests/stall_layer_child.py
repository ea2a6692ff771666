"""Child process of test_failure_layers_gpu.py (run as a script, never collected by pytest).

It starts with GLA_TEST_STALL_ONE_LOAD set, so the first call of this process leaves out the load of one chunk: that
call must report GLA_ERR_DEVICE_TIMEOUT after its bounded waits run out, and the same call, once more, must match its
64-bit form. The argument names the call. Prints one JSON line with what it saw.
"""
import json
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import layer_ref as ref  # noqa: E402


def scan(backward, splits):
    """The call, and what it has to give."""
    from chunkwise_recurrent_prefill_gb300 import ssm_bwd, ssm_fwd
    from test_ssm_gpu import GRADS, make
    d = make(2, 100, 40, 1, 16, "f32", seed=6)
    t = {n: ref.gpu(v) for n, v in d.items()}
    a = (t["u"], t["dt"], t["A"], t["Bm"], t["Cm"])
    k = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h0=t["h0"], seq_splits=splits)

    def run():
        if backward:
            return dict(zip(GRADS, ssm_bwd(t["do"], *a, dhT=t["dhT"], **k)))
        return dict(zip(("o", "hT"), ssm_fwd(*a, return_state=True, **k)))

    return run, ref.scan(d, back=backward)


CALLS = {"scan": lambda: scan(False, 1), "scan in segments": lambda: scan(False, 2), "scan gradients": lambda: scan(True, 1)}


def main():
    import torch
    from chunkwise_recurrent_prefill_gb300 import last_device_status
    assert os.environ.get("GLA_TEST_STALL_ONE_LOAD")
    run, want = CALLS[sys.argv[1]]()
    torch.cuda.synchronize()
    out = {"status_before": last_device_status()}
    t0 = time.time()
    run()
    out["status_stalled"] = last_device_status()
    out["waited_s"] = time.time() - t0
    out["status_cleared"] = last_device_status()
    for n, v in run().items():
        ref.close(n, v, *want[n])
    out["status_after"] = last_device_status()
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
