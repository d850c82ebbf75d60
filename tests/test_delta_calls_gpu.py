"""Calls of the gated delta rule that its other tests leave out."""
import pytest
import torch

import delta_testutil as du
from test_delta_gpu import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    import selective_state_space_05_gb300 as m
    return m


def split(d):
    d = du.to(d, "cuda")
    return tuple(d[n] for n in du.NAMES), dict(initial_states=d["initial_states"],
                                               seq_idx=d["seq_idx"])


def run_bwd(saved, dout, ins, init, dfinal, dinit):
    """ssd_delta_scan_bwd with d_initial_states where the caller says."""
    from selective_state_space_05_gb300 import _lib
    lib = _lib.load()
    q, k, v, g, beta = ins
    (B, L, G, K), (H, V) = q.shape, v.shape[2:]
    dt = _lib.SSD_DTYPE_BF16 if q.dtype is BF else _lib.SSD_DTYPE_F32
    n = lib.ssd_delta_scan_bwd_workspace_bytes(B, L, H, V, K, G, dt, 1, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in ins]
    st = [x for t in (q, k, v) for x in (t.data_ptr(), _lib.Stride(t.stride(0), t.stride(1)))]
    code = lib.ssd_delta_scan_bwd(
        dout.data_ptr(), dfinal.data_ptr(), *st, g.data_ptr(), beta.data_ptr(), K ** -0.5,
        init.data_ptr(), None, B, L, H, V, K, G, dt, saved.data_ptr(), saved.numel(),
        *(t.data_ptr() for t in out), dinit.data_ptr(), ws.data_ptr(), n,
        torch.cuda.current_stream().cuda_stream)
    assert code == 0, lib.ssd_last_error()
    return out


@pytest.mark.parametrize("dtype,B,L,H,V,K", [
    (BF, 1, 200, 3, 40, 64), (BF, 4, 1500, 50, 40, 32), (BF, 1, 4101, 2, 200, 128),
    (BF, 1, 1100, 1, 64, 64), (F32, 2, 300, 3, 40, 72)])
def test_states_moved_on_in_place(ssd, dtype, B, L, H, V, K):
    """A prompt in pieces with one tensor for its states, and their gradient: sequences
    in one piece, in segments one after another and in segments all at once."""
    ins, kw = split(du.inputs(B, L, H, H, V, K, dtype, seed=100))
    init = kw["initial_states"]
    out, fin, saved = ssd.delta_scan_fwd(*ins, initial_states=init, return_final_states=True,
                                         save=True)
    dout, df = torch.ones_like(out), torch.randn_like(fin)
    want = torch.empty_like(fin)
    grads = run_bwd(saved, dout, ins, init, df, want)
    for _ in range(5):
        state = init.clone()
        o, s = ssd.delta_scan_fwd(*ins, initial_states=state, final_states=state,
                                  return_final_states=True)
        assert s is state and state._version == 1
        assert torch.equal(o, out) and torch.equal(state, fin)
        state = df.clone()
        got = run_bwd(saved, dout, ins, init, state, state)
        assert torch.equal(state, want)
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
    with pytest.raises(RuntimeError, match="overlaps"):
        ssd.delta_scan_fwd(*ins, out=ins[2])
    with pytest.raises(RuntimeError, match="overlaps"):
        ssd.delta_scan_bwd(dout, *ins, initial_states=init, saved=saved, workspace=saved)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_over_its_values(ssd, dtype):
    d = du.inputs(3, 1, 2, 4, 70, 33, dtype, seed=101)
    ins = [d[n][:, 0].contiguous().cuda() for n in du.NAMES]
    a, b = (d["initial_states"].cuda() for _ in range(2))
    want = ssd.delta_decode_step(*ins, a)
    got = ssd.delta_decode_step(*ins, b, out=ins[2])
    assert got is ins[2] and torch.equal(got, want) and torch.equal(a, b)
    with pytest.raises(RuntimeError, match="overlaps"):
        ssd.delta_decode_step(*ins, b, out=b.view(dtype).flatten()[:3 * 4 * 70].view(3, 4, 70))


TOP = 3.4e38    # finite in fp32, an infinity where it is rounded to bf16


def large(dtype, L, where):
    """Keys and queries along the axes in turn, a weak decay, and one value of TOP (the
    largest of bf16 for tensors of that type): in v, the initial states or a gradient."""
    B, H, V, K = 1, 1, 24, 16
    d = du.inputs(B, L, 1, H, V, K, dtype, seed=110)
    axes = torch.eye(K)[torch.arange(L) % K].view(B, L, 1, K)
    d["q"], d["k"] = axes.to(dtype), axes.roll(1, 1).to(dtype).contiguous()
    d["g"], d["beta"] = torch.full((B, L, H), -1e-3), torch.full((B, L, H), 0.5)
    dout, df = torch.zeros(B, L, H, V), torch.zeros(B, H, V, K)
    top = TOP if dtype is F32 else torch.finfo(BF).max
    if where in ("v", "initial_states"):
        d["v"].zero_()
        d["initial_states"].zero_()
        dout[:, ::7] = 1e-3
        df.fill_(1e-3)
    if where == "v":
        d["v"][0, 5, 0, 3] = top
    elif where == "initial_states":
        d["initial_states"][0, 0, 4, 6] = -TOP
    elif where == "dout":
        dout[0, L - 4, 0, 2] = top
    else:
        df[0, 0, 5, 7] = -TOP
    return d, dout.to(dtype), df


def through(got, ref, dtype, L, what):
    """A state, or its gradient, that has gone through all chunks: with beta = 1/2 each
    visit of an axis halves it, so that a chunk of C tokens leaves 2^-(C / 16) of it,
    by subtracting the rest.  What is subtracted is off by COMPUTE of what the state was
    before, which is 2^(C / 16) times as much of what it is after, in every chunk."""
    C = 64 if dtype is BF else 32
    bound = du.COMPUTE[dtype] * (1 + 2.0 ** (C // 16) * -(-L // C)) * float(ref.norm()) + 1e-30
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    assert float((got - ref).norm()) <= bound, (what, float((got - ref).norm() / ref.norm()))


@pytest.mark.parametrize("dtype,L", [(F32, 40), (F32, 100), (BF, 40), (BF, 150), (BF, 3000)])
@pytest.mark.parametrize("where", ["v", "initial_states", "dout", "dfinal_states"])
def test_finite_values_next_to_infinity(ssd, dtype, L, where):
    """Values that bf16 rounds to an infinity, but fp32 holds, stay finite and keep their
    bits in the states, their gradients and what is computed of them."""
    d, dout, df = large(dtype, L, where)
    if where in ("dout", "dfinal_states"):      # products of two such would overflow
        d["v"] *= 1e-3
        d["initial_states"] *= 1e-3
    ins, kw = split(d)
    want, fin, grads = du.reference(d, dout, df)
    assert max(float(t.abs().max()) for t in (fin, *grads.values())) < 3.4028e38
    out, final, saved = ssd.delta_scan_fwd(*ins, return_final_states=True, save=True, **kw)
    du.close(out, want, dtype, "out")
    through(final, fin, dtype, L, "final_states")
    got = ssd.delta_scan_bwd(dout.cuda(), *ins, saved=saved, dfinal_states=df.cuda(), **kw)
    for n, ref in grads.items():
        if n == "d_initial_states":
            through(got[n], ref, dtype, L, n)
        else:
            du.close(got[n], ref, dtype, n)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_stay_infinite(ssd, dtype):
    """An infinite state or value is no large finite one."""
    for where in ("v", "initial_states"):
        d, _, _ = large(dtype, 100, where)
        for n in ("v", "initial_states"):
            d[n][d[n].abs() > 1e30] = float("inf")
        ins, kw = split(d)
        out, fin = ssd.delta_scan_fwd(*ins, return_final_states=True, **kw)
        row = 3 if where == "v" else 4
        assert not torch.isfinite(fin[0, 0, row]).all()
        assert not torch.isfinite(out[0, 64:, 0, row]).any()
        rest = torch.arange(24, device="cuda") != row
        assert (out[0, :, 0, rest] == 0).all() and (fin[0, 0, rest] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", [1, 40])
def test_decays_beside_a_large_write(ssd, dtype, at):
    """A token whose own write into the final state weighs 2^27 times as much as all
    before it: its decay's gradient is of those before it alone.  Along two axes, in
    powers of two: every product and sum is exact."""
    L = at + 1
    q, k = torch.zeros(1, L, 1, 16), torch.zeros(1, L, 1, 16)
    v, df = torch.zeros(1, L, 1, 8), torch.zeros(1, 1, 8, 16)
    k[0, 0, 0, 0], k[0, at, 0, 1] = 1, 1
    v[0, 0, 0, 0], v[0, at, 0, 0] = 1, 1
    df[0, 0, 0, 0], df[0, 0, 0, 1] = 1, 2.0 ** 27
    g, beta = torch.zeros(1, L, 1), torch.ones(1, L, 1)
    d = dict(q=q, k=k, v=v, g=g, beta=beta, initial_states=None, seq_idx=None)
    _, _, want = du.reference(d, torch.zeros_like(v), df)
    ins = tuple(d[n].to(dtype if n in "qkv" else F32).cuda() for n in du.NAMES)
    got = ssd.delta_scan_bwd(torch.zeros_like(ins[2]), *ins, dfinal_states=df.cuda())
    assert (want["dg"][0, 1:] == 1).all() and want["dg"][0, 0] == 0
    for n in ("dg", "dbeta", "dv"):
        assert torch.equal(got[n].double().cpu(), want[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_workspace_of_another_type_is_kept(ssd, dtype):
    """What the forward returns with save is what the backward takes, when it is the
    caller's own workspace too."""
    ins, kw = split(du.inputs(1, 100, 1, 2, 40, 48, dtype, seed=120))
    out, own = ssd.delta_scan_fwd(*ins, save=True, **kw)
    dout = torch.ones_like(out)
    want = ssd.delta_scan_bwd(dout, *ins, saved=own, **kw)
    ws = torch.empty(-(-own.numel() // 4), device="cuda")
    _, saved = ssd.delta_scan_fwd(*ins, save=True, workspace=ws, **kw)
    assert saved is ws
    got = ssd.delta_scan_bwd(dout, *ins, saved=saved, **kw)
    assert all(torch.equal(got[n], want[n]) for n in want)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        ssd.delta_scan_bwd(dout, *ins, saved=saved[:-64], **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,G,H,V,K", [
    (1, 70, 2, 2, 257, 40), (1, 130, 1, 2, 384, 100), (2, 200, 30, 60, 384, 16),
    (2, 129, 40, 40, 300, 70), (1, 65, 1, 2, 2048, 16), (1, 130, 2, 2, 2048, 128)])
def test_wide_heads(ssd, dtype, B, L, G, H, V, K):
    """More than two blocks of 128 channels, up to the most that is taken; a chunk a CTA
    and several."""
    check(ssd, du.inputs(B, L, G, H, V, K, dtype, seed=V + K), dtype)
