"""The optimizer step's C ABI on the CPU: what it refuses before anything touches a
GPU (the device addresses below are never dereferenced)."""
import ctypes
import math

import pytest

from selective_state_space_05_gb300 import _lib
from selective_state_space_05_gb300.optim import _Options

BF, F32 = _lib.SSD_DTYPE_BF16, _lib.SSD_DTYPE_F32
ARG, NULL, ALIGN, UNSUPPORTED = -1, -2, -3, -4
P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_05_gb300 import build
    build.build()
    return _lib.load()


def arr(t, *v):
    return (t * len(v))(*v)


def test_step_refusals(lib):
    d = dict(p=arr(P, 16, 18), pt=arr(I32, F32, BF), g=arr(P, 16, 18), gt=arr(I32, F32, BF),
             w=None, m=arr(P, 16, 20), v=arr(P, 16, 20), ms=None, vs=None, n=arr(I64, 4, 4),
             count=2, bits=32)

    def f(opt=None, **kw):
        assert not set(kw) - set(d), kw
        o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, max_norm=1.0)
        o.update(opt or {})
        hold = _Options(**o)
        return lib.ssd_adamw_step(*{**d, **kw}.values(), ctypes.addressof(hold), None)

    for o in (dict(beta1=1.0), dict(beta2=-0.5), dict(beta1=math.nan), dict(eps=-1.0),
              dict(eps=math.nan), dict(weight_decay=-1.0), dict(lr=math.inf), dict(lr=math.nan),
              dict(step=0), dict(grad_norm=16, max_norm=-1.0), dict(grad_norm=16, max_norm=math.nan)):
        assert f(o) == ARG, o
    for o in (dict(step_dev=12), dict(lr_dev=18), dict(grad_norm=17)):
        assert f(o) == ALIGN, o
    assert f(count=-1) == ARG and f(bits=16) == ARG and f(n=arr(I64, 4, -1)) == ARG
    assert f(pt=arr(I32, F32, 5)) == ARG and f(gt=arr(I32, 9, BF)) == ARG
    assert f(n=arr(I64, 4, 2 ** 44)) == UNSUPPORTED
    for k in ("p", "pt", "g", "gt", "m", "v", "n"):
        assert f(**{k: None}) == NULL, k
    assert f(bits=8) == NULL and f(bits=8, ms=arr(P, 16, 16), vs=arr(P, 16, None)) == NULL
    for k in ("p", "g", "m", "v"):
        assert f(**{k: arr(P, 16, None)}) == NULL, k
        assert f(**{k: arr(P, 16, 17)}) == ALIGN, k
    assert f(w=arr(P, None, 18)) == ALIGN
    assert f(bits=8, ms=arr(P, 16, 18), vs=arr(P, 16, 16)) == ALIGN
    assert lib.ssd_adamw_step(*d.values(), None, None) == NULL


def test_moments_refusals(lib):
    d = dict(m=arr(P, 17), v=arr(P, 17), ms=arr(P, 16), vs=arr(P, 16), om=arr(P, 16), ov=arr(P, 16),
             n=arr(I64, 4), count=1, stream=None)

    def f(**kw):
        return lib.ssd_adamw_moments(*{**d, **kw}.values())
    assert f(count=-1) == ARG and f(n=arr(I64, -4)) == ARG and f(n=arr(I64, 2 ** 44)) == UNSUPPORTED
    for k in ("m", "v", "ms", "vs", "om", "ov", "n"):
        assert f(**{k: None}) == NULL, k
    for k in ("m", "v", "ms", "vs", "om", "ov"):
        assert f(**{k: arr(P, None)}) == NULL, k
    for k in ("ms", "vs", "om", "ov"):
        assert f(**{k: arr(P, 18)}) == ALIGN, k


def test_version(lib):
    assert lib.ssd_optim_abi_version() == 1


def test_binding_refuses_host_tensors():
    import torch

    import selective_state_space_05_gb300 as ssd
    p = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.adamw_step([p], [p], ssd.adamw_state([p]), step=1, lr=1e-3)
    with pytest.raises(ValueError, match="gradients"):
        ssd.adamw_step([p], [], ssd.adamw_state([p]), step=1, lr=1e-3)
