"""The gated delta rule's C ABI on the CPU: what each call refuses before anything
touches a GPU (the addresses below are never dereferenced), and its workspaces."""
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


IN = dict(q=16, sq=S(64, 16), k=16, sk=S(64, 16), v=16, sv=S(64, 16), g=16, beta=16, scale=0.25,
          init=16, seq=16, batch=2, seqlen=4, nheads=1, headdim=16, dstate=16, ngroups=1, dtype=BF)


def caller(lib, name, **defaults):
    fn = getattr(lib, name)

    def call(**kw):
        assert not set(kw) - set(defaults), kw
        return fn(*{**defaults, **kw}.values())
    return call


def common(f):
    assert f(dtype=7) == ARG and f(batch=0) == ARG and f(seqlen=0) == ARG and f(nheads=0) == ARG
    assert f(headdim=0) == ARG and f(dstate=-1) == ARG and f(ngroups=0) == ARG
    assert f(nheads=3, ngroups=2) == ARG
    assert f(dstate=129) == UNSUPPORTED and f(headdim=2049) == UNSUPPORTED
    assert f(batch=2 ** 20, seqlen=2 ** 20) == UNSUPPORTED and f(seqlen=2 ** 41) == UNSUPPORTED
    assert f(sq=S(-1, 16)) == ARG and f(sv=S(64, -16)) == ARG and f(sk=S(2 ** 41, 1)) == ARG
    assert f(scale=math.nan) == ARG and f(scale=math.inf) == ARG
    for k in ("q", "k", "v", "g", "beta"):
        assert f(**{k: None}) == NULL, k
    assert f(q=17) == ALIGN and f(g=18) == ALIGN and f(init=2) == ALIGN and f(seq=6) == ALIGN
    assert f(dtype=F32, k=18) == ALIGN


def test_forward_refusals(lib):
    f = caller(lib, "ssd_delta_scan_fwd", **IN, out=16, final=16, keep=0, ws=256, wsb=1 << 40,
               stream=None)
    common(f)
    assert f(out=None) == NULL and f(ws=None) == NULL
    assert f(out=17) == ALIGN and f(final=18) == ALIGN and f(ws=128) == ALIGN
    ws = lib.ssd_delta_scan_workspace_bytes(2, 4, 1, 16, 16, 1, BF, 0, 1)
    assert f(wsb=ws - 1) == WORKSPACE and b"workspace" in lib.ssd_last_error()
    kept = lib.ssd_delta_scan_workspace_bytes(2, 4, 1, 16, 16, 1, BF, 1, 1)
    assert kept > ws > 0 and f(keep=1, wsb=kept - 1) == WORKSPACE
    assert lib.ssd_delta_scan_workspace_bytes(2, 0, 1, 16, 16, 1, BF, 0, 1) == 0
    assert lib.ssd_delta_scan_workspace_bytes(2, 4, 1, 16, 129, 1, BF, 0, 1) == 0


def test_backward_refusals(lib):
    f = caller(lib, "ssd_delta_scan_bwd", dout=16, dfinal=16, **IN, saved=256, sb=1 << 40, dq=16,
               dk=16, dv=16, dg=16, dbeta=16, dinit=16, ws=256, wsb=1 << 40, stream=None)
    common(f)
    for k in ("dout", "dq", "dk", "dv", "dg", "dbeta", "ws"):
        assert f(**{k: None}) == NULL, k
    assert f(dout=17) == ALIGN and f(dq=18) == ALIGN and f(dinit=2) == ALIGN
    assert f(saved=16) == ALIGN and f(ws=16) == ALIGN
    q = lib.ssd_delta_scan_bwd_workspace_bytes
    own, whole = (q(2, 4, 1, 16, 16, 1, BF, s, 1) for s in (1, 0))
    kept = lib.ssd_delta_scan_workspace_bytes(2, 4, 1, 16, 16, 1, BF, 1, 1)
    assert whole == own + kept
    assert f(sb=kept - 1) == WORKSPACE and f(wsb=own - 1) == WORKSPACE
    assert f(saved=None, wsb=whole - 1) == WORKSPACE
    assert q(2, 4, 3, 16, 16, 2, BF, 1, 1) == 0
    # rows off 16 bytes are copied where the kernels read by tensor maps
    wide = q(2, 4, 1, 64, 16, 1, BF, 1, 1)
    assert q(2, 4, 1, 64, 16, 1, BF, 1, 0) >= wide + 2 * 4 * (2 * 16 + 2 * 64) * 2
    assert q(2, 4, 1, 64, 16, 1, F32, 1, 0) == q(2, 4, 1, 64, 16, 1, F32, 1, 1)


def test_step_refusals(lib):
    f = caller(lib, "ssd_delta_decode_step", q=16, k=16, v=16, g=16, beta=16, scale=1.0, state=16,
               batch=2, nheads=2, headdim=8, dstate=8, ngroups=1, dtype=BF, out=16, stream=None)
    assert f(dtype=3) == ARG and f(batch=0) == ARG and f(ngroups=3) == ARG
    assert f(dstate=129) == UNSUPPORTED and f(headdim=4000) == UNSUPPORTED
    assert f(batch=2 ** 31) == UNSUPPORTED and f(scale=math.nan) == ARG
    for k in ("q", "k", "v", "g", "beta", "state", "out"):
        assert f(**{k: None}) == NULL, k
    assert f(v=17) == ALIGN and f(state=18) == ALIGN


def test_version(lib):
    assert lib.ssd_delta_abi_version() == 1


def test_binding_refuses_host_tensors():
    import torch

    import selective_state_space_05_gb300 as ssd
    q, g = torch.zeros(1, 2, 1, 8), torch.zeros(1, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_scan_fwd(q, q, q, g, g)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ssd.delta_scan(q.half(), q, q, g, g)
