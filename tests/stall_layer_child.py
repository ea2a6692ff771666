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

import torch  # noqa: E402

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


def qk(backward):
    from chunkwise_recurrent_prefill_gb300 import qk_norm_bwd, qk_norm_fwd
    g = torch.Generator().manual_seed(7)
    B, T, D = 2, 50, 64
    q, dq = ref.draw(g, B, T, 4, D), ref.draw(g, B, T, 4, D)
    k, dk = ref.draw(g, B, T, 2, D), ref.draw(g, B, T, 2, D)
    wq, wk = ref.draw(g, D), ref.draw(g, D)
    angle = torch.rand(T, D // 2, generator=g) * 6
    cos, sin, positions = torch.cos(angle), torch.sin(angle), torch.arange(T).expand(B, T)
    t = [ref.gpu(x) for x in (q, k, wq, wk)]
    kw = dict(cos=cos.cuda(), sin=sin.cuda())
    # the forward's factors to 2^-24, which the gradients take as they are
    r = [(x.double().square().mean(-1) + 1e-6).pow(-0.5).float() for x in (q, k)]

    def run():
        if backward:
            out = qk_norm_bwd(dq.cuda(), dk.cuda(), *t[:2], r[0].cuda(), r[1].cuda(), *t[2:], **kw)
            return dict(zip(("dx0", "dx1", "dw0", "dw1"), out))
        return dict(zip(("out0", "out1", "r0", "r1"), qk_norm_fwd(*t, **kw)))

    want = {}
    for i, (x, w, go) in enumerate(((q, wq, dq), (k, wk, dk))):
        for n, v in ref.qk(x, w, cos, sin, positions, "rms", False, 1e-6, go, r[i]).items():
            want[f"{n}{i}"] = v
    return run, want


CALLS = {"scan": lambda: scan(False, 1), "scan in segments": lambda: scan(False, 2), "scan gradients": lambda: scan(True, 1),
         "norm": lambda: qk(False), "norm gradients": lambda: qk(True)}


def main():
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
