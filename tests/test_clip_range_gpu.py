"""Clipping of gradients near the end of fp32's range: the factor keeps its
bits where it is below the smallest normal fp32 value."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_norm", [1.0, 1e-3])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_norm_beyond_the_range(dt, max_norm):
    """Norm 6e39: infinite as an fp32 value, finite in the factor."""
    import selective_state_space_05_gb300 as ssd
    g = torch.Generator().manual_seed(1)
    t = (torch.empty(1003).uniform_(1e38, 3e38, generator=g)).to(dt)
    ref = float(t.double().norm())
    assert ref > torch.finfo(torch.float32).max
    out = torch.empty(1003, device="cuda")
    norm = ssd.clip_grads([t.cuda()], max_norm, out=[out])
    assert float(norm) == float("inf")
    want = t.double() * (max_norm / ref)
    # the norm's error (66, as for other sizes), the factor's and the product's rounding
    bt.assert_within(out, want, want.abs(), 70, "out")
