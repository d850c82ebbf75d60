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


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size,max_norm", [(3e36, 1e-3), (3e36, 1e-10), (9e36, 30.0),
                                           (9e36, 1e37), (1e-3, 1e-38), (1.0, 1e-3)])
def test_clipping_at_the_end_of_the_range(ssd, bits, size, max_norm):
    """The step clips as clip_grads does where the factor or the norm's reciprocal is
    below the normal fp32 range (a norm of 1.6e38 at most here).  Its factor is off by
    three roundings, clip_grads' by one, each of their products by another (two with
    the power of two that keeps its bits); the moment m = (1 - beta1) g' by one more
    each: 9 of 2^-24, where m is a normal number."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    g = [(torch.rand(1000, generator=gen, device="cuda") * 0.9 + 0.1) * size]
    g[0][::2] *= -1
    norm = ssd.grad_norm(g)
    assert torch.isfinite(norm) and float(norm) > max_norm
    clipped = [t.clone() for t in g]
    ssd.clip_grads(clipped, max_norm)
    res = []
    for grads, kw in ((g, dict(grad_norm=norm, max_norm=max_norm)), (clipped, {})):
        p = [torch.zeros(1000, device="cuda")]
        state = ssd.adamw_state(p, bits=bits)
        ssd.adamw_step(p, grads, state, step=1, lr=1.0, betas=(0.5, 0.5), eps=0.0, seed=3, **kw)
        m, v = ssd.adamw_moments(state)
        res.append((m[0].double(), p[0].double(), state))
    (m, p, state), (want, q, other) = res
    if bits == 8:   # (codes are rounded up or down by chance: the blocks' largest are not)
        m, want = (s["exp_avg_scale"][0].double() for s in (state, other))
    small = 2.0 ** -149 if max_norm < 1e-30 else 0.0     # results that are subnormal
    assert ((m - want).abs() <= 9 * 2.0 ** -24 * want.abs() + 4 * small).all(), \
        float(((m - want).abs() / want.abs()).max())
