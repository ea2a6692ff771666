"""Group norm at the edges of its range: means whose square is beyond the largest float, and no values
at all."""
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
