"""Group norm with an activation, channels last, against its 64-bit form.

Bounds. The statistics are fp32 sums of m terms in a tree of partial sums, of deviations from a
mean known to a few u |x|max (u = 2^-24): with k = 2 log2(m) + 32 roundings a statistic is off by
at most k u max(|x|) / std of a unit of x-hat, and so are u and y, times |w| and the activation's
slope (below 1.13). fp32 results are held to 4 k u (1 + |x|max / std) (1 + |value|) |w|max, bf16
ones to 2^-8 of the value more. Channel sums over n rows are held to (log2(n) + 64 + 4 k) u of the
sum of absolute terms.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def act64(act):
    return {"none": lambda t: t, "silu": torch.nn.functional.silu,
            "gelu": torch.nn.functional.gelu}[act]


def reference(x, G, w, b, eps, act, z):
    """y, mean, rstd in float64, differentiable."""
    N, C = x.shape[0], x.shape[-1]
    xg = x.reshape(N, -1, G, C // G)
    mean = xg.mean((1, 3))
    var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    u = (xg - mean[:, None, :, None]) * rstd[:, None, :, None]
    u = u.reshape(x.shape) * w + b
    f = act64(act)
    return (f(u) if z is None else u * f(z)), mean, rstd


def make(shape, io, seed, gate, offset=0.0, strided=False):
    g = torch.Generator("cpu").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    C = shape[-1]

    def draw():
        if strided:
            return torch.randn(*shape[:-1], 3 * C, generator=g).to(dt)[..., C:2 * C]
        return torch.randn(*shape, generator=g).to(dt)

    x = draw()
    x += offset
    return dict(x=x, dy=draw(), z=draw() if gate else None,
                w=1 + 0.3 * torch.randn(C, generator=g), b=0.2 * torch.randn(C, generator=g))


def gpu(t):
    if t is None:
        return None
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return out.copy_(t)


def run(d, G, act, eps=1e-5):
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd, last_device_status
    x, dy, z, w, b = (gpu(d[n]) for n in ("x", "dy", "z", "w", "b"))
    y, mean, rstd = group_norm_fwd(x, G, w, b, eps=eps, act=act, gate=z)
    grads = group_norm_bwd(dy, x, mean, rstd, G, w, b, act=act, gate=z)
    assert last_device_status() == 0
    return y, mean, rstd, grads


def check_all(d, G, act, eps=1e-5):
    y, mean, rstd, (dx, dw, db, dz) = run(d, G, act, eps)
    leaves = {n: d[n].double().requires_grad_() for n in ("x", "w", "b") }
    z = None if d["z"] is None else d["z"].double().requires_grad_()
    ry, rmean, rrstd = reference(leaves["x"], G, leaves["w"], leaves["b"], eps, act, z)
    wrt = [leaves["x"], leaves["w"], leaves["b"]] + ([z] if z is not None else [])
    rg = torch.autograd.grad(ry, wrt, d["dy"].double())
    N, C = d["x"].shape[0], d["x"].shape[-1]
    L = d["x"].numel() // max(N * C, 1)
    m = L * C // G
    k = 2 * math.log2(m) + 32
    xmax = d["x"].double().abs().max().item()
    cond = 1 + xmax * rrstd.max().item()
    wmax = d["w"].abs().max().item()
    bf16 = y.dtype == torch.bfloat16

    def close(name, got, want, factor):
        want = want.detach()
        err = (got.cpu().double() - want).abs()
        bound = 4 * k * U * cond * wmax * factor * (1 + want.abs()) + (2.0 ** -8 * want.abs() if bf16 else 0)
        worst = (err / bound).max().item()
        assert worst <= 1, f"{name}: {worst:.3g} times its bound"

    assert (mean.cpu().double() - rmean).abs().max() <= k * U * (xmax + 1)
    assert ((rstd.cpu().double() - rrstd).abs() / rrstd).max() <= 2 * k * U * cond
    zmax = 1.0 if z is None else 1 + z.detach().abs().max().item()
    close("y", y, ry, zmax)
    dmax = 1 + d["dy"].double().abs().max().item()
    # dx is rstd times a difference of three terms of about dy w
    close("dx", dx, rg[0], rrstd.max().item() * dmax * zmax * (1 + cond * (2 + xmax * rrstd.max().item())))
    if z is not None:
        close("dz", dz, rg[3], dmax * (1 + wmax * 6))
    # channel sums: terms dy act' xhat and dy act'
    f = act64(act)
    xg = d["x"].double().reshape(N, -1, G, C // G)
    xh = ((xg - rmean.detach()[:, None, :, None]) * rrstd.detach()[:, None, :, None]).reshape(d["x"].shape)
    dyz = d["dy"].double().abs() * (1.13 if z is None else f(z.detach()).abs())
    rows = tuple(range(d["x"].dim() - 1))
    s = (math.log2(max(N * L, 2)) + 64 + 4 * k) * U * cond * (1 + wmax)
    for name, got, want, a in (("dw", dw, rg[1], dyz * (xh.abs() + 1)), ("db", db, rg[2], dyz)):
        err = (got.cpu().double() - want).abs()
        bound = s * 4 * (a.sum(rows) + 1)
        assert (err <= bound).all(), f"{name}: {(err / bound).max().item():.3g} times its bound"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape,G", [((5, 64), 4), ((37, 128), 1), ((3, 17, 48), 6), ((2, 9, 7, 40), 5)])
def test_forward_and_gradients(shape, G, act, gate, io):
    check_all(make(shape, io, seed=sum(shape) + G, gate=gate, strided=len(shape) == 3), G, act)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape,G", [
    ((1, 8), 1), ((1, 1, 8), 8), ((700, 2048), 16), ((2, 1000, 64), 32), ((1, 5000, 24), 3),
    ((3, 333, 512), 32), ((4, 50, 7), 7), ((2, 31, 33), 11), ((1, 2, 4096), 1), ((300, 160), 20),
    ((2, 4099, 16), 1), ((9, 3, 1000), 8), ((1, 1200, 1024), 8), ((33, 40, 320), 32)])
def test_sizes(shape, G, io):
    check_all(make(shape, io, seed=shape[0] + shape[-1], gate=shape[0] % 2 == 0), G, "silu")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape,G", [
    ((1, 3000, 72), 9), ((2, 4100, 128), 1),        # clusters of several CTAs in both directions
    ((70, 130, 256), 4), ((3, 2, 16), 1),           # of one
    ((1, 9000, 64), 8), ((1, 20000, 64), 8),        # too long for them: backward, then in both
    ((200, 70, 64), 2), ((500, 40, 512), 8)])       # single CTAs; too many for them
def test_maps_in_clusters_and_in_parts(shape, G, io):
    check_all(make(shape, io, seed=shape[1], gate=shape[0] % 2 == 0), G, "gelu")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape,G", [
    ((900, 320), 32), ((200, 644), 7), ((77, 12), 6),      # per token
    ((3, 2000, 100), 5), ((1, 700, 1284), 3), ((40, 30, 12), 6), ((1, 9000, 60), 6), ((2, 9, 2004), 1)])
def test_groups_that_are_not_whole_vectors(shape, G, gate, io):
    """An even number of channels that is not a multiple of 16 bytes; (2, 9, 2004): too wide for
    anything but the plain kernels."""
    check_all(make(shape, io, seed=shape[-1], gate=gate, strided=True), G, "silu")


@pytest.mark.parametrize("shape,G", [((2, 700, 32), 4), ((50, 256), 2)])
def test_a_mean_far_from_zero(shape, G):
    """The variance of values that all lie near 1000: as a difference of squares it would have no
    digits left."""
    check_all(make(shape, "f32", seed=3, gate=False, offset=1000.0), G, "none")


def test_equal_values_and_eps():
    from chunkwise_recurrent_prefill_gb300 import group_norm_fwd
    x = torch.full((3, 5, 32), 7.25, device="cuda")
    y, mean, rstd = group_norm_fwd(x, 4, eps=1e-3)
    assert torch.equal(mean, torch.full_like(mean, 7.25)) and not y.any()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-3 ** -0.5), rtol=1e-6)


def test_nan_stays_in_its_group():
    from chunkwise_recurrent_prefill_gb300 import group_norm_fwd
    for shape in ((4, 64), (4, 300, 64)):
        x = torch.randn(*shape, device="cuda")
        clean = group_norm_fwd(x, 4)[0]
        x[1, ..., 20] = float("nan")
        x[2, ..., 40] = float("inf")
        y = group_norm_fwd(x, 4)[0]
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[1, ..., 16:32] = True
        bad[2, ..., 32:48] = True
        assert torch.equal(y[~bad], clean[~bad]) and not torch.isfinite(y[1, ..., 16:32]).any()


def test_gradient_against_differences():
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd
    d = make((3, 11, 24), "f32", seed=5, gate=True)
    x, dy, z, w, b = (gpu(d[n]) for n in ("x", "dy", "z", "w", "b"))
    _, mean, rstd = group_norm_fwd(x, 4, w, b, act="gelu", gate=z)
    grads = group_norm_bwd(dy, x, mean, rstd, 4, w, b, act="gelu", gate=z)
    base = {n: d[n].double() for n in ("x", "w", "b", "z")}
    gen = torch.Generator("cpu").manual_seed(6)
    for n, g in zip(("x", "w", "b", "z"), grads):
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-4

        def loss(s):
            a = {**base, n: base[n] + s * h * v}
            y, _, _ = reference(a["x"], 4, a["w"], a["b"], 1e-5, "gelu", a["z"])
            return (y * d["dy"].double()).sum()

        diff = (loss(1) - loss(-1)) / (2 * h)
        dot = (g.cpu().double() * v).sum()
        # fp32 components and an O(h^2) = 1e-8 difference: 1e-5 of the norms
        assert abs(dot - diff) <= 1e-5 * g.double().norm().item() * v.norm()


def test_without_parameters_and_repeated():
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd
    for shape in ((2000, 512), (2, 3000, 64)):
        x = torch.randn(*shape, device="cuda", dtype=torch.bfloat16)
        ones = torch.ones(shape[-1], device="cuda")
        y, mean, rstd = group_norm_fwd(x, 8, act="silu")
        assert torch.equal(y, group_norm_fwd(x, 8, ones, torch.zeros_like(ones), act="silu")[0])
        dx, dw, db, dz = group_norm_bwd(y, x, mean, rstd, 8, act="silu")
        assert dw is None and db is None and dz is None
        full = group_norm_bwd(y, x, mean, rstd, 8, ones, 0 * ones, act="silu")
        again = group_norm_bwd(y, x, mean, rstd, 8, ones, 0 * ones, act="silu")
        assert torch.equal(dx, full[0])
        assert all(torch.equal(p, r) for p, r in zip(full[:3], again[:3]))


def test_empty():
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd
    for shape in ((0, 32), (2, 0, 32)):
        x = torch.zeros(*shape, device="cuda")
        w = torch.ones(32, device="cuda")
        y, mean, rstd = group_norm_fwd(x, 4, w, w)
        assert y.shape == x.shape and mean.shape == (shape[0], 4)
        dx, dw, db, _ = group_norm_bwd(x, x, mean, rstd, 4, w, w)
        assert dx.shape == x.shape and not dw.any() and not db.any()


def test_refusals():
    from chunkwise_recurrent_prefill_gb300 import GLAError, group_norm_bwd, group_norm_fwd
    x = torch.randn(4, 10, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    with pytest.raises(GLAError, match="BAD_SHAPE"):
        group_norm_fwd(x, 5)                                   # 5 does not divide 32
    with pytest.raises(GLAError, match="BAD_SHAPE"):
        group_norm_fwd(x, 0)
    with pytest.raises(GLAError, match="BAD_OPTION"):
        group_norm_fwd(x, 4, eps=-1.0)
    with pytest.raises(ValueError):
        group_norm_fwd(x, 4, act="tanh")
    with pytest.raises(ValueError):
        group_norm_fwd(x.cpu(), 4)
    with pytest.raises(ValueError):
        group_norm_fwd(x.transpose(1, 2), 2)                   # channels not contiguous
    with pytest.raises(ValueError):
        group_norm_fwd(x, 4, w[:16])
    with pytest.raises(TypeError):
        group_norm_fwd(x, 4, w.double())
    with pytest.raises(TypeError):
        group_norm_fwd(x.half(), 4)
    with pytest.raises(TypeError):
        group_norm_fwd(x, 4, gate=x.bfloat16())
    with pytest.raises(GLAError, match="ALIAS"):
        group_norm_fwd(x, 4, y=x)
    with pytest.raises(ValueError):
        group_norm_bwd(x[:2], x, torch.zeros(4, 4, device="cuda"), torch.zeros(4, 4, device="cuda"), 4)
