"""Activations and their derivatives away from the origin: silu' is 1 and 0 far
out."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


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
