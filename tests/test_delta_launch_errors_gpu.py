"""A launch of the gated delta rule or the optimizer step that the driver refuses is
reported by the call that made it.  The refusal is a stream whose graph capture was
invalidated: nothing runs."""
import ctypes

import pytest
import torch

from selective_state_space_05_gb300 import _lib
from selective_state_space_05_gb300.optim import _Options

pytestmark = pytest.mark.gpu

BF, F32 = _lib.SSD_DTYPE_BF16, _lib.SSD_DTYPE_F32
S = _lib.Stride
CUDA_ERROR = -6


def calls(p, ws, st):
    """Small valid arguments in memory at p (each tensor 64 KB) with a workspace of
    4 MB: 2 sequences of 70 tokens, 2 heads of 24 channels, a dstate of 16."""
    a = [p + 65536 * k for k in range(16)]
    n, sizes = 4 << 20, (2, 70, 2, 24, 16, 1)
    ins = (a[0], S(70 * 16, 16), a[1], S(70 * 16, 16), a[2], S(70 * 48, 48), a[3], a[4], 0.25,
           None, None)
    host = {k: (ctypes.c_void_p * 1)(a[k]) for k in range(8)}
    code, size = (ctypes.c_int32 * 1)(F32), (ctypes.c_int64 * 1)(300)
    opt = _Options(beta1=0.9, beta2=0.99, eps=1e-8, lr=1e-3, step=1)
    out = {}
    for name, t in (("bf16", BF), ("fp32", F32)):
        out[f"ssd_delta_scan_fwd {name}"] = (*ins, *sizes, t, a[5], a[6], 1, ws, n, st)
        out[f"ssd_delta_scan_bwd {name}"] = (a[5], None, *ins, *sizes, t, None, 0, *a[6:11], None,
                                             ws, n, st)
        out[f"ssd_delta_decode_step {name}"] = (*a[:5], 0.25, a[5], 2, 2, 24, 16, 1, t, a[6], st)
    out["ssd_adamw_step"] = (host[0], code, host[1], code, None, host[2], host[3], None, None,
                             size, 1, 32, ctypes.addressof(opt), st)
    out["ssd_adamw_moments"] = (*(host[k] for k in range(6)), size, 1, st)
    return out, (opt, host)


@pytest.mark.parametrize("name", calls(0, 0, 0)[0])
def test_a_refused_launch_is_an_error(name):
    lib, drv = _lib.load(), ctypes.CDLL("libcuda.so.1")
    mem = torch.zeros(16 * 65536, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    st = ctypes.c_void_p(stream.cuda_stream)
    table, hold = calls(mem.data_ptr(), ws.data_ptr(), stream.cuda_stream)
    args, call = table[name], getattr(lib, name.split()[0])
    assert call(*args) == 0, lib.ssd_last_error()    # as it is, it runs
    torch.cuda.synchronize()
    assert drv.cuStreamBeginCapture_v2(st, 2) == 0
    try:
        assert drv.cuStreamSynchronize(st) != 0          # not allowed here: the capture is void
        assert call(*args) == CUDA_ERROR
        assert lib.ssd_last_error()
    finally:
        graph = ctypes.c_void_p()
        drv.cuStreamEndCapture(st, ctypes.byref(graph))
    assert call(*args) == 0
    torch.cuda.synchronize()
    del hold
