"""The projections on the GPU, forward and backward, against their 64-bit
definition: sizes on and off the tiles, few rows, split K, strided and
unaligned operands, activations, residuals."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


def _ops(K):
    """fp32 roundings of a sum of K products, in units of the sum of their
    magnitudes: an MMA adds 16 at a time, at most four roundings (or
    truncations, twice as large) a step; then bias, activation (24),
    residual."""
    return 8 * (K // 16 + 1) + 64


def act64(name, v):
    if name == "silu":
        return bt.silu(v)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    return v


CASES = [
    # rows, in, out, dtype, bias, activation, residual dtype
    (1, 8, 8, BF, False, None, None), (1, 64, 1, BF, True, "silu", None),
    (3, 100, 7, BF, True, "gelu", F32), (8, 2560, 1057, BF, False, None, None),
    (16, 264, 333, BF, True, "silu", BF), (17, 64, 64, BF, False, None, None),
    (1, 5, 3, F32, True, "gelu", None), (5, 128, 130, F32, True, None, F32),
    (8, 1000, 67, F32, False, "silu", None), (9, 64, 8, F32, True, None, None),
    (128, 64, 256, BF, False, None, None), (129, 65, 257, BF, True, "silu", BF),
    (200, 2048, 72, BF, True, None, F32), (1000, 520, 1544, BF, True, "gelu", None),
    (300, 1, 5, BF, True, None, None), (257, 7, 130, F32, False, None, None),
    (130, 200, 300, F32, True, "silu", F32), (64, 4096, 24, BF, False, None, None),
    (2000, 72, 640, BF, False, None, F32), (333, 1030, 129, F32, True, "gelu", None),
    (24, 2564, 101, F32, True, "silu", F32), (61, 1024, 1023, F32, True, "gelu", F32),
    (1000, 68, 30, F32, False, None, F32), (700, 1024, 520, F32, True, "silu", None),
]


def _inputs(M, K, N, dt, bias, act, rt, pad=0, seed=0):
    g = torch.Generator().manual_seed(M * 7 + K * 3 + N + seed)
    x = torch.randn(M, K + pad, generator=g).to(dt)
    w = (torch.randn(N, K, generator=g) * K ** -0.5).to(dt)
    b = torch.randn(N, generator=g).to(dt) if bias else None
    r = torch.randn(M, N + pad, generator=g).to(rt) if rt else None
    do = torch.randn(M, N, generator=g).to(rt or dt)
    return x, w, b, r, do


def _c(t):
    return None if t is None else t.cuda()


def _check(M, K, N, dt, act, x, w, b, r, do, out, pre, got):
    X, W = x.double(), w.double()
    p = X @ W.t() + (0 if b is None else b.double())
    pm = X.abs() @ W.abs().t() + (0 if b is None else b.double().abs())
    ref = act64(act, p) + (0 if r is None else r.double())
    # |act'| <= 1.13, so an error of pre comes through at most that much
    mag = 1.13 * pm + (0 if r is None else r.double().abs())
    bt.assert_within(out, ref, mag, _ops(K), "out")
    if got is None:
        return
    P = p.clone().requires_grad_(True)
    dact = torch.autograd.grad(act64(act, P).sum(), P)[0] if act else torch.ones_like(p)
    dp = do.double() * dact
    # errors of dpre: act' of a rounded pre (|act''| <= 0.8), and its rounding
    # to the operands' type
    err = do.double().abs() * (0.8 * pm * _ops(K) * bt.U32 + 64 * bt.U32) if act else 0.0 * pm
    if act and dt == BF:
        err = err + do.double().abs() * 0.8 * p.abs() * 2.0 ** -11 + 2.0 ** -24
    err_op = err
    if dt == BF and (act or do.dtype == F32):
        err_op = err + 2.0 ** -8 * (dp.abs() + err)
    bt.assert_within(got["dx"], dp @ W, dp.abs() @ W.abs(), _ops(N), "dx", err_op @ W.abs())
    bt.assert_within(got["dweight"], dp.t() @ X, dp.abs().t() @ X.abs(), _ops(M), "dweight",
                     err_op.t() @ X.abs())
    if got["dbias"] is not None:
        bt.assert_within(got["dbias"], dp.sum(0), dp.abs().sum(0), M + 64, "dbias", err.sum(0))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_linear(case):
    import selective_state_space_05_gb300 as ssd
    M, K, N, dt, bias, act, rt = case
    x, w, b, r, do = _inputs(*case)
    cx, cw, cb, cr, cdo = map(_c, (x, w, b, r, do))
    out, pre = ssd.linear_fwd(cx, cw, cb, activation=act, residual=cr, save_pre=True)
    assert out.dtype == (rt or dt) and pre.dtype == (torch.float16 if dt == BF else F32)
    got = ssd.linear_bwd(cdo, cx, cw, activation=act, pre=pre, need_dbias=bias)
    ssd.scan_status()
    _check(M, K, N, dt, act, x, w, b, r, do, out, pre, got)


# rows, in, out that the product kernel cuts differently: single CTAs and pairs,
# tiles 32 to 256 wide, one to sixteen splits of K, several rounds of tiles and of splits,
# sums in one run and in several (an fp32 residual keeps the sum exact)
TILES = [(700, 512, 1500), (2500, 640, 700), (3000, 4096, 520), (260, 8192, 264),
         (513, 2048, 1032), (100, 2100, 4200), (5000, 136, 5000), (40, 24000, 40),
         (1999, 1000, 3001), (611, 2100, 3591)]


@pytest.mark.parametrize("rt", [None, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", TILES, ids=str)
def test_tiles(shape, dt, rt):
    import selective_state_space_05_gb300 as ssd
    M, K, N = shape
    g = torch.Generator("cuda").manual_seed(M + K + N)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, w, b = r(M, K).to(dt), (r(N, K) * K ** -0.5).to(dt), r(N).to(dt)
    res = None if rt is None else r(M, N)
    do = r(M, N).to(rt or dt)
    out = ssd.linear_fwd(x, w, b, residual=res)
    got = ssd.linear_bwd(do, x, w, need_dbias=True)
    ssd.scan_status()
    X, W, D = x.double(), w.double(), do.double()
    ref, mag = X @ W.t() + b.double(), X.abs() @ W.abs().t() + b.double().abs()
    if res is not None:
        ref, mag = ref + res.double(), mag + res.double().abs()
    bt.assert_within(out, ref.cpu(), mag.cpu(), _ops(K), "out")
    # an fp32 upstream gradient is rounded to bf16 for the two products
    e = 2.0 ** -8 if dt == BF and do.dtype == F32 else 0.0
    for k, v, m, n in (("dx", D @ W, D.abs() @ W.abs(), N), ("dweight", D.t() @ X,
                                                             D.abs().t() @ X.abs(), M)):
        bt.assert_within(got[k], v.cpu(), m.cpu(), _ops(n), k, e * m.cpu())
    bt.assert_within(got["dbias"], D.sum(0).cpu(), D.abs().sum(0).cpu(), M + 64, "dbias")


@pytest.mark.parametrize("case", [(40, 64, 72, BF, True, None, F32), (5, 64, 72, BF, True, None, BF),
                                  (40, 64, 72, F32, False, None, F32), (5, 40, 9, F32, True, None, F32)],
                         ids=str)
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strided_and_unaligned(case, off):
    """x and the residual as slices of wider rows, on and off the 16-byte
    boundaries, give the dense call's values."""
    import selective_state_space_05_gb300 as ssd
    M, K, N, dt, bias, act, rt = case
    x, w, b, r, do = _inputs(*case, pad=16)
    cx, cw, cb, cr, cdo = map(_c, (x, w, b, r, do))
    xs, rs = cx[:, off:off + K], cr[:, off:off + N]
    out = ssd.linear_fwd(xs, cw, cb, residual=rs)
    got = ssd.linear_bwd(cdo, xs, cw, need_dbias=bias)
    ssd.scan_status()
    _check(M, K, N, dt, act, x[:, off:off + K], w, b, r[:, off:off + N], do, out, None, got)
    # the residual's own memory as the output
    dense = rs.contiguous()
    assert torch.equal(ssd.linear_fwd(xs, cw, cb, residual=dense, out=dense), out)
    # a weight and an upstream gradient off the boundary
    wf = torch.empty(N * K + 1, dtype=dt, device="cuda")
    wf[1:] = cw.flatten()
    df = torch.empty(M * N + 1, dtype=cdo.dtype, device="cuda")
    df[1:] = cdo.flatten()
    got2 = ssd.linear_bwd(df[1:].view(M, N), xs, wf[1:].view(N, K), need_dbias=bias)
    assert all(torch.equal(got[k], got2[k]) for k in ("dx", "dweight"))


def test_infinities_stay_in_their_rows():
    import selective_state_space_05_gb300 as ssd
    for dt in (BF, F32):
        x = torch.randn(150, 128, device="cuda").to(dt)
        w = torch.randn(96, 128, device="cuda").to(dt)
        x[7, 5] = float("nan")
        out = ssd.linear_fwd(x, w)
        assert torch.isnan(out[7]).all()
        keep = [i for i in range(150) if i != 7]
        assert torch.isfinite(out[keep]).all()


def test_large_pre_keeps_its_derivative():
    """Beyond the half's range the saved value is the largest half: act' is
    1 or 0 there, not NaN."""
    import selective_state_space_05_gb300 as ssd
    x = torch.full((20, 64), 2.0 ** 8, device="cuda", dtype=BF)
    w = torch.full((16, 64), 2.0 ** 8, device="cuda", dtype=BF)
    w[8:] *= -1
    do = torch.ones(20, 16, device="cuda", dtype=BF)
    for act in ("silu", "gelu"):
        out, pre = ssd.linear_fwd(x, w, activation=act, save_pre=True)
        assert torch.isfinite(pre).all()
        db = ssd.linear_bwd(do, x, w, activation=act, pre=pre, need_dbias=True)["dbias"]
        assert (db[:8] == 20).all() and (db[8:] == 0).all()


def test_differentiable_and_differences():
    import selective_state_space_05_gb300 as ssd
    g = torch.Generator().manual_seed(5)
    x, w, b, r, do = (torch.randn(*s, generator=g).cuda() for s in
                      ((2, 11, 24), (20, 24), (20,), (2, 11, 20), (2, 11, 20)))
    w *= 24 ** -0.5
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b, r)]
    out = ssd.linear(*leaves[:3], activation="gelu", residual=leaves[3])
    grads = torch.autograd.grad(out, leaves, do)
    assert torch.equal(grads[3], do)

    def f(x, w, b, r):
        return float((ssd.linear_fwd(x, w, b, activation="gelu", residual=r).double()
                      * do.double()).sum())

    # h = 2^-6: truncation ~ h^2, rounding of f ~ sqrt(440) 2^-22 / h ~ 4e-4
    for i, gr in enumerate(grads):
        d = torch.randn(gr.shape, generator=torch.Generator().manual_seed(i)).cuda()
        want = float((gr.double() * d.double()).sum())
        got = bt.directional(f, (x, w, b, r), i, d, 2.0 ** -6)
        assert abs(got - want) <= 5e-3 * (1 + float((gr.abs() * d.abs()).sum()) ** 0.5 + abs(want))
    # one gradient alone
    only = torch.autograd.grad(ssd.linear(x, w, leaves[2]), leaves[2], do)[0]
    assert (only - do.sum((0, 1))).abs().max() <= 22 * 2.0 ** -24 * do.abs().sum((0, 1)).max()


def test_streams_graph_and_repeats():
    import selective_state_space_05_gb300 as ssd
    x, w = torch.randn(300, 256, device="cuda").to(BF), torch.randn(512, 256, device="cuda").to(BF)
    do = torch.randn(300, 512, device="cuda").to(BF)

    def step(stream=None):
        out, pre = ssd.linear_fwd(x, w, activation="silu", save_pre=True, stream=stream)
        b = ssd.linear_bwd(do, x, w, activation="silu", pre=pre, stream=stream)
        return out, b["dx"], b["dweight"]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, rec):
        assert torch.equal(a, b) and torch.equal(a, c)
    ssd.scan_status()


def test_refusals():
    import selective_state_space_05_gb300 as ssd
    x, w = torch.zeros(4, 16, device="cuda"), torch.zeros(8, 16, device="cuda")
    with pytest.raises(ValueError, match="activation"):
        ssd.linear_fwd(x, w, activation="relu")
    with pytest.raises(ValueError, match="evenly"):
        ssd.linear_fwd(torch.zeros(4, 6, 16, device="cuda")[:, :5], w)
    with pytest.raises(ValueError, match="dense"):
        ssd.linear_fwd(torch.zeros(16, 4, device="cuda").t(), w)
    with pytest.raises(ValueError, match="weight"):
        ssd.linear_fwd(x, w.to(BF))
    with pytest.raises(ValueError, match="residual"):
        ssd.linear_fwd(x, w, residual=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError, match="pre"):
        ssd.linear_bwd(torch.zeros(4, 8, device="cuda"), x, w, activation="silu")
    with pytest.raises(ssd._lib.SSDError):
        ssd.linear_fwd(x[:0], w)
