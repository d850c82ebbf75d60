"""The differentiable forms of an empty batch: empty results, zero gradients
of the parameters."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


def leaf(*s, dt=F32):
    return torch.randn(*s, device="cuda").to(dt).requires_grad_(True)


@pytest.mark.parametrize("shape", [(0,), (3, 0)])
def test_norms(shape):
    import selective_state_space_05_gb300 as ssd
    x, r, w, sc = leaf(*shape, 16, dt=BF), leaf(*shape, 16), leaf(16), leaf(16)
    y, ro = ssd.add_rmsnorm(x, r, w, scale=sc)
    assert y.shape == ro.shape == (*shape, 16) and (y.dtype, ro.dtype) == (BF, F32)
    (y.float().sum() + ro.sum()).backward()
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
    assert (w.grad == 0).all() and (sc.grad == 0).all()
    y2, ro2 = ssd.add_rmsnorm(x, None, w)
    assert ro2.dtype == BF
    g = ssd.gated_rmsnorm(x, x, w, group_size=8)
    assert g.shape == x.shape and g.dtype == BF
    w.grad = None
    g.float().sum().backward()
    assert (w.grad == 0).all()
    with pytest.raises(ValueError, match="weight"):
        ssd.add_rmsnorm(x, r, leaf(15))
    with pytest.raises(ValueError, match="group_size"):
        ssd.gated_rmsnorm(x, None, w, group_size=5)


@pytest.mark.parametrize("act", [None, "gelu"])
@pytest.mark.parametrize("dt", [F32, BF])
def test_linear(act, dt):
    import selective_state_space_05_gb300 as ssd
    x, w, b = leaf(2, 0, 16, dt=dt), leaf(5, 16, dt=dt), leaf(5, dt=dt)
    r = leaf(2, 0, 5)
    out = ssd.linear(x, w, b, activation=act, residual=r)
    assert out.shape == (2, 0, 5) and out.dtype == F32
    out.sum().backward()
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
    assert (w.grad == 0).all() and w.grad.dtype == dt and (b.grad == 0).all()
    assert ssd.linear(x, w).dtype == dt
    with pytest.raises(ValueError, match="weight"):
        ssd.linear(x, leaf(5, 15, dt=dt))


def test_a_backward_without_upstream_gradients_is_still_checked():
    """Nothing of this changes what the explicit calls refuse."""
    import selective_state_space_05_gb300 as ssd
    x, w = torch.randn(0, 16, device="cuda"), torch.randn(16, device="cuda")
    for call in (lambda: ssd.add_rmsnorm_fwd(x, None, w), lambda: ssd.gated_rmsnorm_fwd(x, None, w),
                 lambda: ssd.linear_fwd(x, w[None])):
        with pytest.raises(ssd._lib.SSDError):
            call()
