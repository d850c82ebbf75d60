"""A projection that takes longer than the limit of one wait inside its kernel
(2 s) is a valid one: its outputs are right and the status says so."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_launch_of_more_than_two_seconds():
    """7.0e15 operations, on 43 + 43 + 54 GB: about 4 s at a library product's
    rate, more than 2 at the tensor cores' own."""
    import selective_state_space_05_gb300 as ssd
    bf = torch.bfloat16
    torch.cuda.empty_cache()
    n, k = 163840, 131072
    x = torch.full((n, k), 0.5, device="cuda", dtype=bf)
    w = torch.full((n, k), 2.0 ** -8, device="cuda", dtype=bf)
    out = torch.empty(n, n, device="cuda", dtype=bf)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    ssd.linear_fwd(x, w, out=out)
    end.record()
    ssd.scan_status()
    assert start.elapsed_time(end) > 2000
    # every block of the output: 2^17 products of 2^-9
    assert (out[::97] == 256).all() and (out[:, ::101] == 256).all()
    del x, w, out
    torch.cuda.empty_cache()
