"""The block's operators past 2^31 elements: the last rows of a large call
equal the same rows in a small one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N = 2 ** 31 + 2 ** 24


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def _big(rows, cols, dtype=BF):
    t = torch.empty(rows, cols, dtype=dtype, device="cuda")
    t[:64].normal_()
    t[64:-64] = 0.5
    t[-64:].normal_()
    return t


def test_norms():
    import selective_state_space_05_gb300 as ssd
    d = 2048
    rows = N // d
    x, w = _big(rows, d), torch.randn(d, device="cuda")
    y, r = ssd.add_rmsnorm_fwd(x, None, w)
    ys, rs = ssd.add_rmsnorm_fwd(x[-64:].clone(), None, w)
    assert torch.equal(y[-64:], ys) and torch.equal(r[-64:], rs)
    got = ssd.add_rmsnorm_bwd(x, None, r, w, need_dresidual=False)
    small = ssd.add_rmsnorm_bwd(x[-64:].clone(), None, rs, w)
    assert torch.equal(got["dx"][-64:], small["dx"])
    del y, r, got
    out = ssd.gated_rmsnorm_fwd(x, x, w, group_size=512)
    assert torch.equal(
        out[-64:], ssd.gated_rmsnorm_fwd(x[-64:].clone(), x[-64:].clone(), w, group_size=512))
    g = ssd.gated_rmsnorm_bwd(x, x, x, w, group_size=512)
    s = ssd.gated_rmsnorm_bwd(*[x[-64:].clone()] * 3, w, group_size=512)
    assert torch.equal(g["dy"][-64:], s["dy"]) and torch.equal(g["dz"][-64:], s["dz"])


def test_conv():
    import selective_state_space_05_gb300 as ssd
    C = 1024
    L = N // C
    x, w = _big(L, C)[None], torch.randn(C, 4, device="cuda")
    g = ssd.causal_conv1d_bwd(x, x, w)
    # the last tokens see 3 before them, and nothing after them
    s = ssd.causal_conv1d_bwd(x[:, -64:].clone(), x[:, -64:].clone(), w)
    assert torch.equal(g["dx"][:, -60:], s["dx"][:, -60:])
    assert torch.isfinite(g["dweight"]).all()


def test_linear():
    import selective_state_space_05_gb300 as ssd
    n, k = 4160, 64
    rows = N // n
    x, w = _big(rows, k), torch.randn(n, k, device="cuda").to(BF)
    res = _big(rows, n)
    out = ssd.linear_fwd(x, w, residual=res, activation="silu")
    small = ssd.linear_fwd(x[-64:].clone(), w, residual=res[-64:].clone(), activation="silu")
    assert (out[-64:].float() - small.float()).abs().max() <= 2 ** -7 * small.float().abs().max()
    # an operand and a gradient of that size
    g = ssd.linear_bwd(res, x, w, need_dbias=True)
    gs = ssd.linear_bwd(res[-64:].clone(), x[-64:].clone(), w)
    assert (g["dx"][-64:].float() - gs["dx"].float()).abs().max() <= (
        2 ** -7 * gs["dx"].float().abs().max())
    want = res[:64].float().sum(0) + res[-64:].float().sum(0) + 0.5 * (rows - 128)
    assert (g["dbias"].float() - want).abs().max() <= 2 ** -7 * want.abs().max()
    ssd.scan_status()


def test_clip():
    import selective_state_space_05_gb300 as ssd
    t = _big(N // 1024, 1024)
    head = torch.randn(5, device="cuda")
    ref = (t[:64].double().square().sum() + t[-64:].double().square().sum()
           + 0.25 * (t.numel() - 128 * 1024) + head.double().square().sum()).sqrt()
    last = t[-1].clone()
    norm = ssd.clip_grads([head, t], float(ref) / 2)
    assert abs(float(norm) - float(ref)) <= 66 * 2.0 ** -24 * float(ref)
    assert torch.equal(t[-1], (last.float() * 0.5).to(BF))
