"""ssd_scan_status costs a process that does not use the gated delta rule nothing more."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
import selective_state_space_05_gb300 as ssd
from torch.profiler import ProfilerActivity, profile

def copies():
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        ssd.scan_status()
        torch.cuda.synchronize()
    return sum("DtoH" in e.name for e in p.events())

x, d = torch.zeros(1, 64, 1, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(1, 64, 1, device="cuda")
torch.ones(1, device="cuda").item()
copies()
ssd.delta_decode_step(x[:, 0], x[:, 0], x[:, 0], d[:, 0], d[:, 0], torch.zeros(1, 1, 64, 64, device="cuda"))
before = copies()
ssd.delta_scan_fwd(x, x, x, d, d)
forward = copies()
ssd.delta_scan_bwd(x, x, x, x, d, d)
print(before, forward, copies())
"""


def test_only_kernels_that_were_launched_are_asked():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    before, forward, backward = map(int, r.stdout.split()[-3:])
    if forward == 0:
        pytest.skip("copies are not traced here")
    # the scan's two words and the projections'; the two of the delta rule's forward; the
    # two of its backward
    assert (before, forward, backward) == (3, 5, 7)
