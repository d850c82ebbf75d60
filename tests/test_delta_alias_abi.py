"""The gated delta rule's C calls refuse outputs that overlap an input or one another,
before anything touches a GPU (the addresses are never dereferenced)."""
import pytest

from selective_state_space_05_gb300 import _lib

ARG, M = -1, 1 << 20
F32 = _lib.SSD_DTYPE_F32
S = _lib.Stride
# 2 sequences of 8 tokens, 2 heads of 16 channels, 1 group of 16: tensors in order
# of address, a megabyte apart
SIZES = dict(batch=2, seqlen=8, nheads=2, headdim=16, dstate=16, ngroups=1, dtype=F32)
QK, V, STATE, GATE = 2 * 8 * 16 * 4, 2 * 8 * 32 * 4, 2 * 2 * 16 * 16 * 4, 2 * 8 * 2 * 4


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_05_gb300 import build
    build.build()
    return _lib.load()


def inputs():
    return dict(q=1 * M, sq=S(128, 16), k=2 * M, sk=S(128, 16), v=3 * M, sv=S(256, 32), g=4 * M,
                beta=5 * M, scale=0.25, init=6 * M, seq=7 * M, **SIZES)


def check(f, base, outs, ins, allowed=()):
    """Each output at each input's first and last bytes; the outputs pairwise.  Both
    are at most a megabyte."""
    def refused(**kw):
        return f({**base, **kw}) == ARG
    for o, no in outs.items():
        for i, ni in ins.items():
            if (o, i) not in allowed:
                assert refused(**{o: base[i]}), (o, i)
            assert refused(**{o: base[i] + ni // 256 * 256 - 256}) or ni < 512, (o, i)
            if base[i] >= no and no >= 512:
                assert refused(**{o: base[i] - no // 256 * 256 + 256}), (o, i)
        for p in outs:
            assert p == o or refused(**{o: base[p]}), (o, p)


def test_forward(lib):
    base = dict(inputs(), out=8 * M, final=9 * M, keep=0, ws=16 * M, wsb=1 << 40, stream=None)
    ws = lib.ssd_delta_scan_workspace_bytes(2, 8, 2, 16, 16, 1, F32, 0, 1)
    check(lambda d: lib.ssd_delta_scan_fwd(*d.values()), base,
          dict(out=V, final=STATE, ws=ws),
          dict(q=QK, k=QK, v=V, g=GATE, beta=GATE, init=STATE, seq=64), {("final", "init")})
    # views of a wide projection: their last token is far behind the first
    wide = dict(base, sv=S(8 * M, M), v=32 * M)
    assert lib.ssd_delta_scan_fwd(*dict(wide, out=32 * M + 4 * (15 * M) + 64).values()) == ARG
    assert lib.ssd_last_error().startswith(b"an output overlaps")


def test_backward(lib):
    base = dict(dout=17 * M, dfinal=18 * M, **inputs(), saved=20 * M, sb=1 << 40, dq=8 * M,
                dk=9 * M, dv=10 * M, dg=11 * M, dbeta=12 * M, dinit=13 * M, ws=30 * M,
                wsb=1 << 40, stream=None)
    kept = lib.ssd_delta_scan_workspace_bytes(2, 8, 2, 16, 16, 1, F32, 1, 1)
    own = lib.ssd_delta_scan_bwd_workspace_bytes(2, 8, 2, 16, 16, 1, F32, 1, 1)
    check(lambda d: lib.ssd_delta_scan_bwd(*d.values()), base,
          dict(dq=QK, dk=QK, dv=V, dg=GATE, dbeta=GATE, dinit=STATE, ws=own),
          dict(q=QK, k=QK, v=V, g=GATE, beta=GATE, init=STATE, seq=64, dout=V, dfinal=STATE,
               saved=kept), {("dinit", "dfinal")})


def test_step(lib):
    base = dict(q=1 * M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, scale=1.0, state=6 * M, batch=64,
                nheads=2, headdim=16, dstate=16, ngroups=1, dtype=F32, out=8 * M, stream=None)
    n = 64
    check(lambda d: lib.ssd_delta_decode_step(*d.values()), base,
          dict(out=n * 32 * 4, state=n * 512 * 4),
          dict(q=n * 64, k=n * 64, v=n * 128, g=n * 8, beta=n * 8), {("out", "v")})
