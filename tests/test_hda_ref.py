"""The 64-bit forms of the decay attention against brute force and against differences (CPU)."""
import torch

from hda_ref import backward, forward, inputs


def test_forward_is_the_decayed_sum():
    x = inputs(2, 9, 4, 4, 2, 1, 8, 16, "f32", seed=1)
    o, hT = forward(x["q"], x["k"], x["v"], x["decay"], 0.5, x["h0"])
    b, h, t = 1, 3, 6
    q, k, v = (x[n][b].double() for n in "qkv")
    lam = torch.exp(x["decay"].double())[h]
    ref = lam ** (t + 1) * q[t, 3] @ x["h0"][b, h].double()
    for j in range(t + 1):
        ref = ref + lam ** (t - j) * (q[t, 3] @ k[j, 1]) * v[j, 0]
    assert torch.allclose(o[b, t, h], 0.5 * ref, rtol=1e-12, atol=1e-12)
    S = lam ** 9 * x["h0"][b, h].double()
    for j in range(9):
        S = S + lam ** (8 - j) * k[j, 1][:, None] * v[j, 0][None, :]
    assert torch.allclose(hT[b, h], S, rtol=1e-12, atol=1e-12)


def test_gradients_against_differences():
    """The loss is linear in each argument alone, so a central difference is exact."""
    x = inputs(2, 7, 4, 2, 4, 1, 8, 8, "f32", seed=2)
    args = {n: x[n].double() for n in ("q", "k", "v", "h0")}

    def loss(**kw):
        a = {**args, **kw}
        o, hT = forward(a["q"], a["k"], a["v"], x["decay"], 0.7, a["h0"])
        return (o * x["do"].double()).sum() + (hT * x["dhT"].double()).sum()

    grads = backward(x["do"], x["q"], x["k"], x["v"], x["decay"], 0.7, x["h0"], x["dhT"])
    gen = torch.Generator("cpu").manual_seed(3)
    for n, g in zip(("q", "k", "v", "h0"), grads):
        d = torch.randn(args[n].shape, generator=gen, dtype=torch.float64)
        diff = (loss(**{n: args[n] + d}) - loss(**{n: args[n] - d})) / 2
        assert torch.allclose((g * d).sum(), diff, rtol=1e-10)
