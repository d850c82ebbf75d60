"""Activations and their derivatives away from the origin: fp32 results keep
fp32 accuracy where the sigmoid is small, and silu' is 1 and 0 far out."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16

# fp32 roundings of silu(v) = v * sigmoid(v): the argument's, the exponential
# (2 units of 2^-23), 1 +, the reciprocal (1 unit), the product: below 12
SILU = 12


def far(n=512):
    """Values over [-85, 85], where sigmoid and its exponential are normal."""
    return torch.linspace(-85.0, 85.0, n)


def silu_terms(v):
    """silu'(v) in 64 bits and the magnitude of its terms."""
    v = v.double()
    s = 1 / (1 + torch.exp(-v))
    c = 1 / (1 + torch.exp(v))          # 1 - s without cancellation
    return s * (1 + v * c), s * (1 + v.abs() * (c + 2.0 ** -1))


def test_silu_of_the_projection():
    import selective_state_space_05_gb300 as ssd
    b = far()
    w = torch.zeros(512, 64, device="cuda")
    for rows in (3, 200):
        x = torch.zeros(rows, 64, device="cuda")
        out = ssd.linear_fwd(x, w, b.cuda(), activation="silu")
        ref = bt.silu(b.double()).expand(rows, -1)
        bt.assert_within(out, ref, ref.abs(), SILU, f"{rows} rows")


def test_derivatives_of_the_projection():
    import selective_state_space_05_gb300 as ssd
    w = torch.zeros(512, 8, device="cuda")
    x = torch.zeros(1, 8, device="cuda")
    one = torch.ones(1, 512, device="cuda")
    v = far()
    for act in ("silu", "gelu"):
        if act == "gelu":
            v = torch.linspace(-12.0, 12.0, 512)
        got = ssd.linear_bwd(one, x, w, activation=act, pre=v.cuda()[None], need_dbias=True)
        d = v.double()
        if act == "silu":
            ref, mag = silu_terms(v)
        else:
            tail = d * torch.exp(-0.5 * d * d) * (2 * torch.pi) ** -0.5
            ref = 0.5 * torch.erfc(-d * 0.5 ** 0.5) + tail
            # 1 + erf is rounded at its 1; the exponential's argument, up to 72,
            # in proportion to it
            mag = torch.maximum(torch.ones_like(d) * 0.5, tail.abs() * (1 + d * d / 8))
        bt.assert_within(got["dbias"], ref, mag, 2 * SILU, act)


def test_gate():
    """Groups of eight equal channels: the norm is that of a constant."""
    import selective_state_space_05_gb300 as ssd
    z = far()[:, None].expand(-1, 8).contiguous()
    y, w = torch.full_like(z, 1.5), torch.ones(8)
    out = ssd.gated_rmsnorm_fwd(y.cuda(), z.cuda(), w.cuda(), eps=0.0, norm_before_gate=True)
    ref = bt.gated_rmsnorm(y.double(), z.double(), w.double(), 8, 0.0, True)
    # the norm: squares and their sum (8), the mean, the root (2 units), the products
    bt.assert_within(out, ref, ref.abs(), SILU + 16, "out")


def test_conv():
    import selective_state_space_05_gb300 as ssd
    b = far()
    zero, w = torch.zeros(1, 512, device="cuda"), torch.zeros(512, 4, device="cuda")
    state = torch.zeros(1, 3, 512, device="cuda")
    out = ssd.causal_conv1d_step(zero, state, w, b.cuda())
    ref = bt.silu(b.double())[None]
    bt.assert_within(out, ref, ref.abs(), SILU, "step")
    x = zero.expand(5, -1).contiguous()[None]
    got = ssd.causal_conv1d_bwd(torch.ones_like(x), x, w, b.cuda())
    ref, mag = silu_terms(b)
    bt.assert_within(got["dbias"], 5 * ref, 5 * mag, 2 * SILU, "dbias")


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("before", [False, True])
def test_large_gates_keep_their_derivative(dt, before):
    """silu' is 1 for large z, also where z + 1 is not a value of the type,
    and 0 for large negative z."""
    import selective_state_space_05_gb300 as ssd
    size = torch.tensor([2.0 ** k for k in range(4, 40)])
    z = torch.cat([size, -size])[:, None].expand(-1, 8).contiguous().to(dt)
    g = torch.Generator().manual_seed(1)
    y = (torch.randn(72, 8, generator=g)).to(dt)
    do, w = torch.randn(72, 8, generator=g).to(dt), torch.randn(8, generator=g)
    eps = 1e-5
    got = ssd.gated_rmsnorm_bwd(do.cuda(), y.cuda(), z.cuda(), w.cuda(), eps=eps,
                                norm_before_gate=before)
    Y, Z, W, D = (t.double() for t in (y, z, w, do))
    s, c = 1 / (1 + torch.exp(-Z)), 1 / (1 + torch.exp(Z))
    e, de = Z * s, s * (1 + Z * c)
    u = Y if before else Y * e
    r = 1 / (u.square().mean(-1, keepdim=True) + eps).sqrt()
    gr = W * D * (e if before else 1.0)
    if before:
        dz, mag = W * D * Y * r * de, (W * D * Y * r * de).abs()
    else:
        du = r * (gr - u * r * r * (gr * u).mean(-1, keepdim=True))
        dm = r * (gr.abs() + u.abs() * r * r * (gr * u).abs().mean(-1, keepdim=True))
        dz, mag = du * Y * de, dm * (Y * de).abs()
    # 1.2 |z| roundings of the exponential where bf16 instances take the short one
    ops = 128 if dt == F32 else 128 + 1.2 * 128
    bt.assert_within(got["dz"], dz, mag, ops, "dz")
