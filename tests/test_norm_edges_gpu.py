"""Group norm at the edges of its range: means whose square is beyond the largest float, no values at
all, and gradients that their mean terms make up."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# clusters of several CTAs, of one, too long for them in both directions
MAPS = [((1, 3000, 72), 9), ((3, 2, 16), 1), ((70, 130, 256), 4), ((1, 20000, 64), 8), ((500, 40, 512), 8),
        ((3, 2000, 100), 5)]


@pytest.mark.parametrize("value", [1e20, -3e30])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,G", MAPS)
def test_equal_values_beyond_the_root_of_the_range(shape, G, io, value):
    """A constant map has no variance, whatever its value: y = b, and dx = (du w - mean) / sqrt(eps)."""
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd
    C = shape[-1]
    x = torch.full(shape, value, device="cuda", dtype=io)
    gen = torch.Generator("cuda").manual_seed(1)
    w, b = (torch.randn(C, device="cuda", generator=gen) for _ in range(2))
    dy = torch.randn(*shape, device="cuda", generator=gen).to(io)
    y, mean, rstd = group_norm_fwd(x, G, w, b, eps=1.0)
    assert torch.equal(mean, torch.full_like(mean, x.flatten()[0].item()))
    assert torch.equal(rstd, torch.ones_like(rstd))
    assert torch.equal(y, b.to(io).expand_as(y))
    dx, dw, db, _ = group_norm_bwd(dy, x, mean, rstd, G, w, b)
    assert not dw.any() and torch.isfinite(db).all()
    d = (dy.double() * w.double()).view(shape[0], -1, G, C // G)
    want = (d - d.mean((1, 3), keepdim=True)).view(shape)
    # the mean of up to 10^5 terms and three roundings of terms of 5 or so, and bf16's own
    tol = 1e-5 + (2.0 ** -8 * want.abs() if io == torch.bfloat16 else 0)
    assert ((dx.double() - want).abs() <= tol).all()


def test_statistics_of_no_values():
    """mean and rstd of no positions are the formula's 0 / 0, not what the memory held."""
    from chunkwise_recurrent_prefill_gb300 import group_norm_fwd
    for shape in ((2, 0, 32), (3, 4, 0, 8)):
        held = [torch.full((shape[0], 4), 7.0, device="cuda") for _ in range(4)]
        del held        # (what the allocator hands out again)
        _, mean, rstd = group_norm_fwd(torch.zeros(*shape, device="cuda"), 4)
        assert mean.shape == rstd.shape == (shape[0], 4)
        assert mean.isnan().all() and rstd.isnan().all()


# ---------------------------------------------------------------- the gradient's mean terms
def mean_terms(shape, io, seed):
    """Inputs whose mean(du w) and mean(du w xhat) are about 1: dy is a constant, the value itself
    and noise."""
    g = torch.Generator("cpu").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    C = shape[-1]
    x = torch.randn(*shape, generator=g)
    dy = 1.5 + 1.5 * x + torch.randn(*shape, generator=g)
    return dict(x=x.to(dt), dy=dy.to(dt), w=1 + 0.1 * torch.randn(C, generator=g),
                b=0.1 * torch.randn(C, generator=g))


def gradients64(d, G, terms=(1, 1)):
    """dx, dw, db by the formula in float64; terms: how often each mean is subtracted."""
    x, dy, w = (d[n].double() for n in ("x", "dy", "w"))
    N, C = x.shape[0], x.shape[-1]
    xg = x.reshape(N, -1, G, C // G)
    rstd = 1 / ((xg - xg.mean((1, 3), keepdim=True)).square().mean((1, 3), keepdim=True) + 1e-5).sqrt()
    xh = (xg - xg.mean((1, 3), keepdim=True)) * rstd
    u = xh.reshape(x.shape) * w + d["b"].double()
    s = torch.sigmoid(u)
    du = dy * s * (1 + u * (1 - s))
    dxh = (du * w).reshape(xg.shape)
    dx = rstd * (dxh - terms[0] * dxh.mean((1, 3), keepdim=True)
                 - terms[1] * xh * (dxh * xh).mean((1, 3), keepdim=True))
    rows = tuple(range(x.dim() - 1))
    return dx.reshape(x.shape), (du * xh.reshape(x.shape)).sum(rows), du.sum(rows)


def rms(a, b):
    return ((a - b).square().mean() / b.square().mean()).sqrt().item()


# 2^-8 is three times what one rounding to bf16 leaves (2^-9 / sqrt(3)). fp32: x-hat, u, silu', du w,
# the two means and the last three steps are some 20 roundings of 2^-25 rms (2^-24 for the exponential
# and division) of values up to four times the result: 32 x 2^-24 = 2e-6.
BOUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -19}
GRADIENT_SHAPES = MAPS + [((2, 4100, 128), 1), ((1, 9000, 64), 8), ((200, 70, 64), 2), ((2, 1000, 64), 32),
                          ((2, 4099, 16), 1), ((3, 4095, 512), 32), ((700, 2048), 16), ((900, 320), 32),
                          ((33, 33), 11), ((2, 9, 2004), 1)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape,G", GRADIENT_SHAPES)
def test_gradient_whose_mean_terms_count(shape, G, io):
    """Without either mean term, or with one of a cluster's parts left out, dx would be far off."""
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd
    d = mean_terms(shape, io, seed=shape[-1] + G)
    want = gradients64(d, G)
    for without in ((0, 1), (1, 0), (0.9, 1), (1, 0.9)):
        assert rms(gradients64(d, G, without)[0], want[0]) > 4 * BOUND[io], "the input does not tell"
    x, dy, w, b = (d[n].cuda() for n in ("x", "dy", "w", "b"))
    _, mean, rstd = group_norm_fwd(x, G, w, b, act="silu")
    got = group_norm_bwd(dy, x, mean, rstd, G, w, b, act="silu")
    for name, g, r in zip(("dx", "dw", "db"), got, want):
        e = rms(g.cpu().double(), r)
        # (sums of channels are fp32 whatever the tensors are)
        assert e <= (BOUND[io] if name == "dx" else BOUND["f32"] * (1 if io == "f32" else 4)), f"{name}: {e:.3g}"


@pytest.mark.parametrize("shape,G", [((1, 3000, 72), 9), ((1, 20000, 64), 8), ((500, 40, 512), 8)])
def test_gradient_against_differences_over_several_ctas(shape, G):
    """A direction with a mean and a part along x-hat. fp32 components, and a central difference in 64
    bits (h = 1e-4 squared): 1e-5 of the norms."""
    from chunkwise_recurrent_prefill_gb300 import group_norm_bwd, group_norm_fwd
    d = mean_terms(shape, "f32", seed=G)
    x, dy, w, b = (d[n].cuda() for n in ("x", "dy", "w", "b"))
    _, mean, rstd = group_norm_fwd(x, G, w, b, act="silu")
    dx = group_norm_bwd(dy, x, mean, rstd, G, w, b, act="silu")[0].cpu().double()
    x64, gen = d["x"].double(), torch.Generator("cpu").manual_seed(7)
    N, C = shape[0], shape[-1]

    def loss(t):
        xg = t.reshape(N, -1, G, C // G)
        m = xg.mean((1, 3), keepdim=True)
        u = ((xg - m) / ((xg - m).square().mean((1, 3), keepdim=True) + 1e-5).sqrt()).reshape(shape)
        return (torch.nn.functional.silu(u * d["w"].double() + d["b"].double()) * d["dy"].double()).sum()

    for v in (torch.ones(shape, dtype=torch.float64), x64.clone(),
              torch.randn(shape, generator=gen, dtype=torch.float64)):
        diff = (loss(x64 + 1e-4 * v) - loss(x64 - 1e-4 * v)) / 2e-4
        assert abs((dx * v).sum() - diff) <= 1e-5 * dx.norm() * v.norm()
