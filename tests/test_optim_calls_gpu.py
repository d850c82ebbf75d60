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


def test_another_shape(ssd):
    """A gradient, moment or master of as many elements in another shape."""
    def dense(*shape):
        return torch.ones(shape, device="cuda")
    p, g = [dense(8, 4).to(torch.bfloat16), dense(3)], [dense(8, 4), dense(3)]
    for bits in (32, 8):
        good = ssd.adamw_state(p, bits=bits, master=True)
        with pytest.raises(ValueError, match="grads"):
            ssd.adamw_step(p, [dense(4, 8), g[1]], good, step=1, lr=1e-3)
        for name in ("exp_avg", "exp_avg_sq", "master"):
            bad = dict(good, **{name: [good[name][0].view(4, 8), good[name][1]]})
            with pytest.raises(ValueError, match=name):
                ssd.adamw_step(p, g, bad, step=1, lr=1e-3)
        if bits == 8:
            with pytest.raises(ValueError, match="out"):
                ssd.adamw_moments(good, out=([dense(4, 8), dense(3)], [dense(8, 4), dense(3)]))
        assert all((t == 1).all() for t in p)
        ssd.adamw_step(p, g, good, step=1, lr=0.0)
        assert all((t == 1).all() for t in p)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_of_the_state_twice(ssd, bits):
    """Two parameters with one moment, scale or master, or one tensor for both moments:
    two threads would write the same element."""
    p = [torch.zeros(300, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    g = [torch.ones(300, device="cuda") for _ in range(2)]
    good = ssd.adamw_state(p, bits=bits, master=True)
    for name, ts in good.items():
        with pytest.raises(ValueError, match="twice"):
            ssd.adamw_step(p, g, dict(good, **{name: [ts[0], ts[0]]}), step=1, lr=1e-3)
    if bits == 32:
        with pytest.raises(ValueError, match="twice"):
            ssd.adamw_step(p, g, dict(good, exp_avg_sq=good["exp_avg"]), step=1, lr=1e-3)
        with pytest.raises(ValueError, match="twice"):
            ssd.adamw_step(p, g, dict(good, master=good["exp_avg"][::-1]), step=1, lr=1e-3)
    assert all((t == 0).all() for t in p)
    # without elements, or without masters, nothing is written twice
    none = [torch.zeros(0, device="cuda") for _ in range(2)]
    ssd.adamw_step(none, none, ssd.adamw_state(none, bits=bits), step=1, lr=1e-3)
    ssd.adamw_step(p, g, dict(good, master=[None, None]), step=1, lr=0.0)
