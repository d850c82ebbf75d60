"""A launch that the driver refuses is reported by the call that made it.  The
refusal is a stream whose graph capture was invalidated: nothing runs."""
import ctypes

import pytest
import torch

from selective_state_space_05_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = _lib.SSD_DTYPE_BF16, _lib.SSD_DTYPE_F32
S = _lib.Stride
CUDA_ERROR = -6


def calls(p, ws, st):
    """Every call of the block's operators, on small valid arguments in memory
    at p (each tensor 64 KB) with a workspace of 1 MB."""
    a, b, c, d, e, f, g, h, i = (p + 65536 * k for k in range(9))
    host = (ctypes.c_void_p * 1)(a), (ctypes.c_int64 * 1)(64), (ctypes.c_int32 * 1)(F32)
    n = 1 << 20
    return {
        "ssd_add_rmsnorm_fwd": (a, b, None, c, 1e-5, 4, 8, BF, F32, d, e, st),
        "ssd_add_rmsnorm_bwd": (a, b, c, d, e, f, 1e-5, 4, 8, BF, F32, g, h, i, i, ws, n, st),
        "ssd_gated_rmsnorm_fwd": (a, S(32, 8), b, S(32, 8), c, 1e-5, 2, 4, 8, 8, 0, BF, d, st),
        "ssd_gated_rmsnorm_bwd": (a, b, S(32, 8), c, S(32, 8), d, 1e-5, 2, 4, 8, 8, 0, BF, e, f,
                                  S(32, 8), g, ws, n, st),
        "ssd_causal_conv1d_bwd": (a, S(64, 16), b, S(64, 16), c, d, None, 2, 4, 16, 4, 1, BF, e,
                                  S(64, 16), f, g, ws, n, st),
        "ssd_causal_conv1d_step": (a, 16, b, c, None, 2, 16, 4, 1, BF, d, st),
        "ssd_linear_fwd": (a, 64, b, None, None, 0, 4, 64, 32, 0, BF, BF, c, None, ws, n, st),
        "ssd_linear_bwd": (a, BF, b, 64, c, None, 40, 64, 32, 0, BF, d, e, f, ws, n, st),
        "ssd_grad_norm": (*host, 1, b, ws, n, st),
        "ssd_clip_grads": (*host, 1, None, None, 1.0, 0.0, b, ws, n, st),
    }


@pytest.mark.parametrize("name", calls(0, 0, 0))
def test_a_refused_launch_is_an_error(name):
    lib, drv = _lib.load(), ctypes.CDLL("libcuda.so.1")
    mem = torch.zeros(9 * 65536, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    st = ctypes.c_void_p(stream.cuda_stream)
    args = calls(mem.data_ptr(), ws.data_ptr(), stream.cuda_stream)[name]
    assert getattr(lib, name)(*args) == 0    # as it is, it runs
    torch.cuda.synchronize()
    assert drv.cuStreamBeginCapture_v2(st, 2) == 0
    try:
        assert drv.cuStreamSynchronize(st) != 0          # not allowed here: the capture is void
        assert getattr(lib, name)(*args) == CUDA_ERROR
        assert lib.ssd_last_error()
    finally:
        graph = ctypes.c_void_p()
        drv.cuStreamEndCapture(st, ctypes.byref(graph))
    assert getattr(lib, name)(*args) == 0
    torch.cuda.synchronize()
