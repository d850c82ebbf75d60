"""Calls of the gated delta rule that its other tests leave out."""
import pytest
import torch

import delta_testutil as du

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
