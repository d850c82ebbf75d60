"""The block operators' C ABI on the CPU: what each call refuses, before
anything touches a GPU (the addresses below are never dereferenced), and the
workspace queries."""
import math

import pytest

from selective_state_space_05_gb300 import _lib

BF, F32 = _lib.SSD_DTYPE_BF16, _lib.SSD_DTYPE_F32
ARG, NULL, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -5
S = _lib.Stride


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_05_gb300 import build
    build.build()
    return _lib.load()


def caller(lib, name, **defaults):
    fn = getattr(lib, name)

    def call(**kw):
        assert not set(kw) - set(defaults), kw
        return fn(*{**defaults, **kw}.values())
    return call


def test_block_abi_version(lib):
    assert lib.ssd_block_abi_version() == 1


def test_add_rmsnorm_refusals(lib):
    f = caller(lib, "ssd_add_rmsnorm_fwd", x=16, residual=16, scale=None, weight=16, eps=1e-5,
               rows=4, dim=8, dtype=BF, rdtype=F32, y=16, rout=16, stream=None)
    assert f(dtype=9) == ARG and f(rdtype=-1) == ARG
    assert f(dtype=F32, rdtype=BF) == ARG and b"fp32 residual" in lib.ssd_last_error()
    assert f(rows=0) == ARG and f(dim=0) == ARG and f(rows=-3) == ARG
    assert f(eps=-1.0) == ARG and f(eps=math.nan) == ARG
    assert f(rows=2 ** 31) == UNSUPPORTED and f(dim=16385) == UNSUPPORTED
    for k in ("x", "weight", "y", "rout"):
        assert f(**{k: None}) == NULL, k
    assert f(x=17) == ALIGN and f(residual=18) == ALIGN and f(weight=6) == ALIGN
    ws = lib.ssd_add_rmsnorm_bwd_workspace_bytes(4, 8)
    assert ws >= 4 * 2 * 8 * 4 and ws % 256 == 0
    assert lib.ssd_add_rmsnorm_bwd_workspace_bytes(0, 8) == 0
    assert lib.ssd_add_rmsnorm_bwd_workspace_bytes(4, 16385) == 0
    b = caller(lib, "ssd_add_rmsnorm_bwd", dy=16, dro=16, ro=16, x=16, scale=16, weight=16,
               eps=1e-5, rows=4, dim=8, dtype=BF, rdtype=F32, dx=16, dres=16, dw=16, ds=16,
               ws=256, wsb=1 << 20, stream=None)
    assert b(rows=0) == ARG and b(dim=16385) == UNSUPPORTED
    for k in ("dy", "ro", "weight", "dw", "ws", "ds", "x"):
        assert b(**{k: None}) == NULL, k
    assert b(scale=None) == NULL            # dscale without scale
    assert b(ws=128) == ALIGN and b(dy=1) == ALIGN and b(dres=2) == ALIGN
    assert b(wsb=ws - 1) == WORKSPACE


def test_gated_rmsnorm_refusals(lib):
    f = caller(lib, "ssd_gated_rmsnorm_fwd", y=16, ys=S(32, 8), z=16, zs=S(32, 8), weight=16,
               eps=1e-5, batch=2, seqlen=4, dim=8, gs=8, before=0, dtype=BF, out=16, stream=None)
    assert f(dtype=5) == ARG and f(gs=3) == ARG and f(gs=0) == ARG and f(seqlen=0) == ARG
    assert f(batch=0) == ARG and f(eps=-0.5) == ARG
    assert f(ys=S(-1, 8)) == ARG and f(zs=S(32, -8)) == ARG
    assert f(batch=2 ** 20, seqlen=2 ** 11) == UNSUPPORTED
    assert f(dim=16392, gs=16392) == UNSUPPORTED and f(dim=65536, gs=1) == UNSUPPORTED
    for k in ("y", "weight", "out"):
        assert f(**{k: None}) == NULL, k
    assert f(z=17) == ALIGN
    ws = lib.ssd_gated_rmsnorm_bwd_workspace_bytes(2, 4, 8, 8)
    assert ws > 0 and lib.ssd_gated_rmsnorm_bwd_workspace_bytes(2, 4, 8, 3) == 0
    b = caller(lib, "ssd_gated_rmsnorm_bwd", dout=16, y=16, ys=S(32, 8), z=16, zs=S(32, 8),
               weight=16, eps=1e-5, batch=2, seqlen=4, dim=8, gs=8, before=0, dtype=BF, dy=16,
               dz=16, dzs=S(32, 8), dw=16, ws=256, wsb=1 << 20, stream=None)
    assert b(gs=3) == ARG and b(dzs=S(32, 4)) == ARG and b(dzs=S(4, 8)) == ARG
    for k in ("dout", "y", "weight", "dy", "dw", "ws", "z", "dz"):
        assert b(**{k: None}) == NULL, k
    assert b(ws=16) == ALIGN and b(wsb=ws - 1) == WORKSPACE


def test_binding_refuses_host_tensors():
    import torch

    import selective_state_space_05_gb300 as ssd
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.add_rmsnorm_fwd(x, None, w)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ssd.gated_rmsnorm_fwd(x.half(), None, w)


def test_conv_refusals(lib):
    d = dict(dout=16, dos=S(64, 16), x=16, xs=S(64, 16), weight=16, bias=16, seq=16, batch=2,
             seqlen=4, channels=16, width=4, silu=1, dtype=BF, dx=16, dxs=S(64, 16), dw=16, db=16,
             ws=256, wsb=1 << 20, stream=None)
    f = caller(lib, "ssd_causal_conv1d_bwd", **d)
    assert f(dtype=2) == ARG and f(batch=0) == ARG and f(seqlen=0) == ARG and f(batch=65536) == ARG
    assert f(channels=12) == UNSUPPORTED and f(width=9) == UNSUPPORTED and f(width=0) == UNSUPPORTED
    for k in ("dout", "x", "weight", "dx", "dw", "ws"):
        assert f(**{k: None}) == NULL, k
    assert f(x=8) == ALIGN and f(dx=24) == ALIGN and f(ws=16) == ALIGN
    assert f(xs=S(64, 20)) == ALIGN and f(dos=S(64, 8)) == ALIGN and f(dxs=S(60, 16)) == ALIGN
    assert f(dxs=S(0, 16)) == ARG
    ws = lib.ssd_causal_conv1d_bwd_workspace_bytes(2, 4, 16, 4)
    assert ws >= 2 * 16 * 5 * 4 and f(wsb=ws - 1) == WORKSPACE
    assert lib.ssd_causal_conv1d_bwd_workspace_bytes(2, 4, 12, 4) == 0
    g = caller(lib, "ssd_causal_conv1d_step", x=16, xs=16, state=16, weight=16, bias=None, batch=2,
               channels=16, width=4, silu=1, dtype=BF, out=16, stream=None)
    assert g(batch=0) == ARG and g(channels=4) == UNSUPPORTED and g(width=9) == UNSUPPORTED
    for k in ("x", "state", "weight", "out"):
        assert g(**{k: None}) == NULL, k
    assert g(x=8) == ALIGN and g(xs=20) == ALIGN and g(state=24) == ALIGN


def test_clip_refusals(lib):
    import ctypes

    def arr(t, *v):
        return (t * len(v))(*v)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    d = dict(g=arr(P, 16, 18), n=arr(I64, 4, 4), gt=arr(I32, F32, BF), count=2, outs=None, ot=None,
             max_norm=1.0, eps=1e-6, norm=16, ws=256, wsb=1 << 20, stream=None)
    f = caller(lib, "ssd_clip_grads", **d)
    assert f(count=-1) == ARG and f(max_norm=-1.0) == ARG and f(max_norm=math.nan) == ARG
    assert f(eps=-1.0) == ARG and f(n=arr(I64, 4, -1)) == ARG and f(gt=arr(I32, F32, 7)) == ARG
    assert f(n=arr(I64, 4, 2 ** 45)) == UNSUPPORTED
    for k in ("g", "n", "gt", "norm", "ws"):
        assert f(**{k: None}) == NULL, k
    assert f(g=arr(P, 16, None)) == NULL
    assert f(outs=arr(P, 16, None)) == NULL
    assert f(g=arr(P, 18, 18)) == ALIGN and f(g=arr(P, 16, 17)) == ALIGN
    assert f(outs=arr(P, 16, 18), ot=arr(I32, F32, F32)) == ALIGN
    assert f(norm=18) == ALIGN and f(ws=16) == ALIGN
    ws = lib.ssd_clip_grads_workspace_bytes(2)
    assert f(wsb=ws - 1) == WORKSPACE and lib.ssd_clip_grads_workspace_bytes(-1) == 0
    assert lib.ssd_clip_grads_workspace_bytes(2000) > ws


def test_linear_refusals(lib):
    d = dict(x=16, sx=64, weight=16, bias=16, res=16, sr=32, rows=40, k=64, n=32, act=0, dtype=BF,
             rdtype=F32, out=16, pre=None, ws=256, wsb=1 << 30, stream=None)
    f = caller(lib, "ssd_linear_fwd", **d)
    assert f(dtype=3) == ARG and f(act=3) == ARG and f(act=-1) == ARG
    assert f(rows=0) == ARG and f(k=0) == ARG and f(n=-1) == ARG
    assert f(dtype=F32, rdtype=BF) == ARG
    assert f(sx=63) == ARG and f(sr=31) == ARG and f(sx=2 ** 41) == ARG
    assert f(rows=2 ** 31) == UNSUPPORTED and f(k=2 ** 25) == UNSUPPORTED
    assert f(rows=2 ** 30, n=2 ** 24) == UNSUPPORTED
    for k in ("x", "weight", "out"):
        assert f(**{k: None}) == NULL, k
    assert f(x=17) == ALIGN and f(bias=17) == ALIGN and f(res=18) == ALIGN and f(pre=17) == ALIGN
    assert f(ws=128) == ALIGN
    # operands that are laid out in the workspace need it
    assert f(x=18, wsb=0) == WORKSPACE and f(x=18, ws=None) == NULL
    q = lib.ssd_linear_fwd_workspace_bytes
    assert q(0, 64, 32, BF, 1) == 0 and q(40, 64, 32, 9, 1) == 0
    big = 40000   # enough rows for no split
    assert q(big, 64, 256, BF, 1) == 0 and q(8, 64, 256, BF, 1) == 0
    assert q(big, 64, 256, BF, 0) >= (big * 64 + 256 * 64) * 2
    assert q(big, 65, 256, BF, 1) >= (big + 256) * 72 * 2
    assert q(big, 64, 256, F32, 1) >= 3 * (big + 256) * 64 * 2
    b = caller(lib, "ssd_linear_bwd", dout=16, ddt=BF, x=16, sx=64, weight=16, pre=None, rows=40,
               k=64, n=32, act=0, dtype=BF, dx=16, dw=16, db=16, ws=256, wsb=1 << 30, stream=None)
    assert b(ddt=7) == ARG and b(dtype=F32, ddt=BF) == ARG and b(act=4) == ARG and b(rows=0) == ARG
    assert b(sx=60) == ARG
    for k in ("dout", "x", "weight", "ws"):
        assert b(**{k: None}) == NULL, k
    assert b(act=1) == NULL                       # an activation needs pre
    assert b(dout=17) == ALIGN and b(dw=1) == ALIGN and b(ws=64) == ALIGN
    assert b(wsb=16) == WORKSPACE
    assert lib.ssd_linear_bwd_workspace_bytes(40, 64, 32, BF, 1, 1) > 0
    assert lib.ssd_linear_bwd_workspace_bytes(40, 0, 32, BF, 1, 1) == 0
