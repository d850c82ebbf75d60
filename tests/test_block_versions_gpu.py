"""Calls that write into a given tensor tell autograd so: a value saved for a
backward pass and overwritten since is an error, not a wrong gradient."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _t(*s):
    return torch.randn(*s, device="cuda")


def test_versions_move_on():
    import selective_state_space_05_gb300 as ssd
    x, r, w = _t(4, 16), _t(4, 16), _t(16)
    o = _t(4, 16)
    ssd.add_rmsnorm_fwd(x, r, w, out=o, residual_out=r)
    assert (x._version, r._version, o._version) == (0, 1, 1)
    ssd.gated_rmsnorm_fwd(x, r, w, out=o)
    assert o._version == 2
    z = _t(4, 16)
    ssd.gated_rmsnorm_bwd(x, x, r, w, dz=z)
    assert z._version == 1 and x._version == 0
    ssd.linear_fwd(x, _t(16, 16), residual=r, out=r)
    assert r._version == 2
    state = _t(4, 3, 16)
    cw = _t(16, 4)
    ssd.causal_conv1d_step(x, state, cw, out=o)
    assert state._version == 1 and o._version == 3 and x._version == 0
    x3, dx = _t(2, 5, 16), _t(2, 5, 16)
    ssd.causal_conv1d_bwd(x3, x3, cw, dx=dx)
    assert dx._version == 1 and x3._version == 0
    a, b = _t(7), _t(3, 2)
    ssd.grad_norm([a, b])
    assert a._version == b._version == 0
    into = [_t(7), _t(3, 2)]
    ssd.clip_grads([a, b], 0.5, out=into)
    assert a._version == 0 and into[0]._version == into[1]._version == 1
    ssd.clip_grads([a, b], 0.5)
    assert a._version == b._version == 1


def test_overwritten_values_are_noticed():
    import selective_state_space_05_gb300 as ssd
    x, w = _t(4, 16), _t(16)
    leaf = _t(4, 16).requires_grad_(True)
    r = leaf * 1.0
    loss = (r * r).sum()                        # saves r
    with torch.no_grad():
        ssd.add_rmsnorm_fwd(x, r.detach(), w, residual_out=r.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_under_inference_mode():
    import selective_state_space_05_gb300 as ssd
    with torch.inference_mode():
        x, r, w = _t(4, 16), _t(4, 16), _t(16)
        ssd.add_rmsnorm_fwd(x, r, w, residual_out=r)
        ssd.clip_grads([x], 1.0)
