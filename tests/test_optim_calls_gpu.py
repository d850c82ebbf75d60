"""Calls of the optimizer's step that its other tests leave out."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def ssd():
    import selective_state_space_05_gb300 as m
    return m


def test_scales_that_are_not_dense(ssd):
    """Refused in both calls: the kernels read one scale after another."""
    p, g = [torch.zeros(600, device="cuda")], [torch.ones(600, device="cuda")]
    wide = torch.zeros(3, 2, device="cuda")
    for name in ("exp_avg_scale", "exp_avg_sq_scale"):
        for bad in (wide[:, 0], torch.zeros(1, device="cuda").expand(3)):
            state = ssd.adamw_state(p, bits=8)
            state[name] = [bad]
            with pytest.raises(ValueError, match="dense"):
                ssd.adamw_step(p, g, state, step=1, lr=1e-3)
            with pytest.raises(ValueError, match="dense"):
                ssd.adamw_moments(state)
    assert (p[0] == 0).all()
