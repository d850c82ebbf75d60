"""The causal conv1d's backward and its one-token step on the GPU against the
definition in 64 bits."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16

# fp32 roundings of a value: the window's sum (8 + 1), the sigmoid (its
# exponential 2 + 1.16 |pre|, |pre| < 12, its division: 20), silu' (4), and the
# sum of dx over the window (8): about 45
OPS = 64


def conv(x, w, b, seq):
    """The definition: taps of the same document and sequence only."""
    B, L, C = x.shape
    W = w.shape[1]
    out = torch.zeros_like(x) + (0 if b is None else b)
    for k in range(W):
        lag = W - 1 - k
        if lag >= L:
            continue
        tap = x[:, :L - lag] * w[:, k]
        if seq is not None:
            tap = torch.where((seq[:, lag:] == seq[:, :L - lag])[..., None], tap,
                              torch.zeros_like(tap))
        out = out + torch.nn.functional.pad(tap, (0, 0, lag, 0))
    return out


CASES = [
    # batch, seqlen, channels, width, dtype, elements before / after, documents, silu, bias
    (1, 1, 8, 4, F32, 0, 0, None, True, True), (2, 3, 16, 4, BF, 8, 8, None, True, True),
    (1, 2, 8, 8, F32, 4, 0, None, True, False), (1, 517, 128, 4, BF, 0, 0, [100, 1, 2, 300, 114],
                                                 True, True),
    (3, 130, 40, 2, F32, 4, 4, None, False, True), (2, 200, 40, 7, F32, 4, 0, [63, 64, 73], True,
                                                    True),
    (2, 97, 264, 3, BF, 16, 24, [1] * 97, True, True), (1, 4000, 520, 4, BF, 8, 0, None, True,
                                                        True),
    (4, 333, 1032, 1, BF, 0, 0, None, True, True), (1, 1000, 24, 5, F32, 0, 0, [999, 1], True,
                                                    True),
    (2, 64, 32, 6, BF, 0, 0, [31, 33], False, False),
]


def _inputs(B, L, C, W, dt, before, after, lens, silu, bias):
    g = torch.Generator().manual_seed(L * 3 + C + W)
    src = torch.randn(B, L, before + C + after, generator=g).to(dt)
    dsrc = torch.randn(B, L, after + C, generator=g).to(dt)
    w = torch.randn(C, W, generator=g) * 0.5
    b = torch.randn(C, generator=g) * 0.3 if bias else None
    seq = None
    if lens:
        seq = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(lens)])
        seq = seq.unsqueeze(0).expand(B, -1).contiguous()
    return src, dsrc, w, b, seq


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:7]))
def test_causal_conv1d_bwd(case):
    import selective_state_space_05_gb300 as ssd
    B, L, C, W, dt, before, after, lens, silu, bias = case
    src, dsrc, w, b, seq = _inputs(*case)
    x, dout = src[..., before:before + C], dsrc[..., after:]
    cx, cdo = src.cuda()[..., before:before + C], dsrc.cuda()[..., after:]
    if after * cdo.element_size() % 16:
        cdo = cdo.contiguous()
    buf = torch.full_like(src, 5.0).cuda()
    got = ssd.causal_conv1d_bwd(cdo, cx, w.cuda(), None if b is None else b.cuda(),
                                seq_idx=None if seq is None else seq.cuda(),
                                activation="silu" if silu else None,
                                dx=buf[..., before:before + C])
    X, Wt, Bs = bt.leaf(x), bt.leaf(w), bt.leaf(b)
    pre = conv(X, Wt, Bs, seq)
    y = bt.silu(pre) if silu else pre
    leaves = [t for t in (X, Wt, Bs) if t is not None]
    grads = torch.autograd.grad(y, leaves, dout.double())
    # magnitudes: the same gradients of the conv's adjoint with every term
    # positive (dpre's own error grows with the terms of pre)
    with torch.no_grad():
        pm = conv(X.abs(), Wt.abs(), None if Bs is None else Bs.abs(), seq)
        dpm = dout.double().abs() * ((bt.dsilu_mag(pre) + 0.5 * pm) if silu else 1.0)
    Xa, Wa = bt.leaf(x.abs()), bt.leaf(w.abs())
    mags = torch.autograd.grad(conv(Xa, Wa, None, seq), (Xa, Wa), dpm)
    bt.assert_within(got["dx"], grads[0], mags[0], OPS, "dx")
    # a sum's chain: a range's tokens, then the ranges (152 x 8 at most) in 8 rows
    ops = OPS + L + 152 + 8
    bt.assert_within(got["dweight"], grads[1], mags[1], ops, "dweight")
    if bias:
        bt.assert_within(got["dbias"], grads[2], dpm.sum((0, 1)), ops, "dbias")
    else:
        assert got["dbias"] is None
    assert (buf[..., :before] == 5).all() and (buf[..., before + C:] == 5).all()


def test_other_documents_do_not_leak():
    """NaN and infinity in one document stay there, forward and backward."""
    import selective_state_space_05_gb300 as ssd
    x = torch.randn(1, 40, 8, device="cuda")
    do = torch.randn(1, 40, 8, device="cuda")
    seq = (torch.arange(40, device="cuda", dtype=torch.int32) >= 17).int()[None].contiguous()
    w, b = torch.randn(8, 4, device="cuda"), torch.randn(8, device="cuda")
    x[0, 16], do[0, 15] = float("inf"), float("nan")
    got = ssd.causal_conv1d_bwd(do, x, w, b, seq_idx=seq)
    assert torch.isfinite(got["dx"][0, 17:]).all() and torch.isfinite(got["dx"][0, :12]).all()
    assert torch.isnan(got["dx"][0, 12:16]).any()


def test_differentiable_and_differences():
    import selective_state_space_05_gb300 as ssd
    g = torch.Generator().manual_seed(3)
    x, w, b, do = (torch.randn(*s, generator=g).cuda() for s in ((2, 21, 16), (16, 4), (16,),
                                                                 (2, 21, 16)))
    plain = ssd.causal_conv1d(x, w, b)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    out = ssd.causal_conv1d(*leaves)
    assert torch.equal(out.detach(), plain) and out.requires_grad
    grads = torch.autograd.grad(out, leaves, do)

    def f(x, w, b):
        return float((ssd.causal_conv1d(x, w, b).double() * do.double()).sum())

    # h = 2^-7: truncation ~ h^2, rounding of f ~ sqrt(672) 2^-24 / h ~ 2e-4
    for i, gr in enumerate(grads):
        d = torch.randn(gr.shape, generator=torch.Generator().manual_seed(i)).cuda()
        want = float((gr.double() * d.double()).sum())
        got = bt.directional(f, (x, w, b), i, d, 2.0 ** -7)
        assert abs(got - want) <= 5e-3 * (1 + float((gr.abs() * d.abs()).sum()) ** 0.5 + abs(want))


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("B,C,W", [(1, 8, 1), (3, 40, 2), (8, 5376, 4), (70, 520, 8)])
def test_step_continues_the_forward(dt, B, C, W):
    """Tokens fed one by one, each a strided slice, give the forward's outputs
    and leave its last inputs."""
    import selective_state_space_05_gb300 as ssd
    L = 6
    g = torch.Generator().manual_seed(C + W)
    x = torch.randn(B, L, C, generator=g).to(dt).cuda()
    w, b = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    want = ssd.causal_conv1d(x, w, b)
    state = torch.zeros(B, W - 1, C, dtype=dt, device="cuda")
    for t in range(L):
        out = ssd.causal_conv1d_step(x[:, t], state, w, b)
        ref = bt.silu(conv(x[:, :t + 1].double().cpu(), w.double().cpu(), b.double().cpu(),
                           None)[:, -1])
        mag = conv(x[:, :t + 1].double().cpu().abs(), w.double().cpu().abs(),
                   b.double().cpu().abs(), None)[:, -1]
        bt.assert_within(out, ref, mag, OPS, f"token {t}")
        assert (out.float() - want[:, t].float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
        last = x[:, max(0, t - W + 2):t + 1]
        assert torch.equal(state[:, W - 1 - last.shape[1]:], last[:, :W - 1])
