"""The residual RMSNorm and the gated grouped RMSNorm on the GPU, forward and
backward, against their 64-bit definitions, at the sizes, types, strides and
values where they can go wrong."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16

# fp32 roundings an element may have seen: inputs combined (3), the in-thread
# chain of a row's sum (8 x 4), shuffles (5), warps (32), rsqrt and division
# (4), products (6), a sigmoid (2 + 1.16 |z| of its exponential, |z| < 6,
# twice, and its division: 20): about 100; one power of two above.
OPS = 128


def _sum_ops(rows):
    """Column sums: a term's own error, the chain of rows of a team (at least
    152 x 4 / 8 teams walk the rows) and of the teams' partial sums."""
    return OPS + rows // 76 + 1 + 152 * 4 * 4 // 8 + 8


ADD_CASES = [
    # rows, dim, x dtype, residual dtype (None: no residual), scale
    (1, 1, F32, F32, False), (1, 7, BF, F32, True), (3, 8, BF, BF, True), (5, 64, F32, F32, True),
    (33, 100, BF, BF, False), (2, 257, F32, None, True), (8, 2560, BF, F32, False),
    (700, 2560, BF, F32, True), (9, 4104, F32, F32, True), (3, 8200, BF, F32, True),
    (2, 16384, BF, BF, True), (2, 16383, F32, F32, False), (2000, 24, BF, F32, True),
]


def _add_inputs(rows, dim, dt, rt, scale, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 31 + dim)
    x = torch.randn(rows, dim, generator=g).to(dt)
    res = None if rt is None else (torch.randn(rows, dim, generator=g) * 3).to(rt)
    w = torch.randn(dim, generator=g) * 0.3 + 1
    sc = torch.randn(dim, generator=g) * 0.5 if scale else None
    rt = rt or dt
    dy = torch.randn(rows, dim, generator=g).to(dt)
    dr = torch.randn(rows, dim, generator=g).to(rt)
    return x, res, w, sc, dy, dr


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check_add(x, res, w, sc, dy, dr, eps, got_fwd, got):
    X, R, W, S = bt.leaf(x), bt.leaf(res), bt.leaf(w), bt.leaf(sc)
    xs = X.abs() * (1 if sc is None else S.abs())
    mag_r = (xs + (0 if res is None else R.abs())).detach()
    # the norm and the gradients are those of the stored residual: the GPU's
    gy, gr = got_fwd
    bt.assert_within(gr, unrounded(X, R, S), mag_r, 4, "residual_out")
    rs = gr.detach().double().cpu()
    rms = (rs.square().mean(-1, keepdim=True) + eps).sqrt()
    bt.assert_within(gy, w.double() * rs / rms, (w.double() * rs / rms).abs(), OPS, "y")
    if got is None:
        return
    n, g = rs / rms, w.double() * dy.double()
    ref_dr = (g - n * (g * n).mean(-1, keepdim=True)) / rms
    mag = (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True)) / rms
    if dr is not None:
        ref_dr, mag = ref_dr + dr.double(), mag + dr.double().abs()
    s = 1.0 if sc is None else sc.double()
    if got["dresidual"] is not None:
        bt.assert_within(got["dresidual"], ref_dr, mag, OPS, "dresidual")
    bt.assert_within(got["dx"], ref_dr * s, mag * abs(s), OPS, "dx")
    ops = _sum_ops(len(x))
    bt.assert_within(got["dweight"], (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0),
                     ops, "dweight")
    if sc is not None:
        bt.assert_within(got["dscale"], (ref_dr * x.double()).sum(0),
                         (mag * x.double().abs()).sum(0), ops, "dscale")


def unrounded(X, R, S):
    r = X if S is None else X * S
    return (r if R is None else r + R).detach()


@pytest.mark.parametrize("case", ADD_CASES, ids=str)
def test_add_rmsnorm(case):
    import selective_state_space_05_gb300 as ssd
    x, res, w, sc, dy, dr = _add_inputs(*case)
    cx, cres, cw, csc, cdy, cdr = _cuda(x, res, w, sc, dy, dr)
    y, r = ssd.add_rmsnorm_fwd(cx, cres, cw, scale=csc, eps=1e-5)
    assert y.dtype == x.dtype and r.dtype == dr.dtype
    got = ssd.add_rmsnorm_bwd(cdy, cdr, r, cw, x=cx, scale=csc, eps=1e-5)
    _check_add(x, res, w, sc, dy, dr, 1e-5, (y, r), got)
    none = ssd.add_rmsnorm_bwd(cdy, None, r, cw, x=cx, scale=csc, eps=1e-5, need_dresidual=False)
    assert none["dresidual"] is None
    _check_add(x, res, w, sc, dy, None, 1e-5, (y, r), none)


def test_add_rmsnorm_formula_is_its_autograd():
    """The gradient formulas above against autograd of the definition."""
    x, res, w, sc, dy, dr = _add_inputs(4, 33, F32, F32, True)
    X, R, W, S = bt.leaf(x), bt.leaf(res), bt.leaf(w), bt.leaf(sc)
    y, r = bt.add_rmsnorm(X, R, W, S, 1e-5)
    dx, dres, dw, ds = torch.autograd.grad((y, r), (X, R, W, S), (dy.double(), dr.double()))
    rms = (r.square().mean(-1, keepdim=True) + 1e-5).sqrt().detach()
    n, g = r.detach() / rms, w.double() * dy.double()
    ref = dr.double() + (g - n * (g * n).mean(-1, keepdim=True)) / rms
    for a, b in ((dres, ref), (dx, ref * sc.double()), (dw, (dy.double() * n).sum(0)),
                 (ds, (ref * x.double()).sum(0))):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


def test_add_rmsnorm_in_place_and_unaligned_rows():
    import selective_state_space_05_gb300 as ssd
    x, res, w, sc, dy, dr = _add_inputs(17, 64, BF, F32, True)
    flat = torch.zeros(17 * 64 + 1, dtype=BF, device="cuda")
    flat[1:] = x.cuda().flatten()
    cx = flat[1:].view(17, 64)          # off a 16-byte boundary: one element at a time
    cres, cw, csc = _cuda(res, w, sc)
    want = ssd.add_rmsnorm_fwd(x.cuda(), cres, cw, scale=csc)
    y, r = ssd.add_rmsnorm_fwd(cx, cres, cw, scale=csc, residual_out=cres)
    assert r.data_ptr() == cres.data_ptr()
    assert torch.equal(r, want[1])
    _check_add(x, res, w, sc, dy, None, 1e-5, (y, r), None)


def test_add_rmsnorm_zero_rows_and_nan_rows_stay_apart():
    import selective_state_space_05_gb300 as ssd
    x, res, w, _, dy, dr = _add_inputs(6, 40, F32, F32, False)
    x[2], res[2] = 0, 0
    x[4, 3] = float("nan")
    cx, cres, cw, cdy, cdr = _cuda(x, res, w, dy, dr)
    y, r = ssd.add_rmsnorm_fwd(cx, cres, cw)
    got = ssd.add_rmsnorm_bwd(cdy, cdr, r, cw)
    assert torch.equal(y[2], torch.zeros_like(y[2]))
    assert torch.isnan(y[4]).all() and torch.isnan(got["dx"][4]).all()
    keep = [0, 1, 2, 3, 5]
    assert torch.isfinite(y[keep]).all() and torch.isfinite(got["dx"][keep]).all()


def test_add_rmsnorm_autograd_and_differences():
    import selective_state_space_05_gb300 as ssd
    x, res, w, sc, dy, dr = [t.cuda() for t in _add_inputs(5, 96, F32, F32, True)]
    leaves = [t.clone().requires_grad_(True) for t in (x, res, w, sc)]
    y, r = ssd.add_rmsnorm(leaves[0], leaves[1], leaves[2], scale=leaves[3])
    grads = torch.autograd.grad((y, r), leaves, (dy, dr))

    def f(x, res, w, sc):
        y, r = ssd.add_rmsnorm_fwd(x, res, w, scale=sc)
        return float((y.double() * dy.double()).sum() + (r.double() * dr.double()).sum())

    # h = 2^-7: truncation ~ h^2, rounding of f ~ 480 terms * 2^-24 * |y dy| / h ~ 4e-3
    for i, gr in enumerate(grads):
        d = torch.randn(gr.shape, generator=torch.Generator().manual_seed(i)).cuda()
        want = float((gr.double() * d.double()).sum())
        got = bt.directional(f, (x, res, w, sc), i, d, 2.0 ** -7)
        assert abs(got - want) <= 5e-3 * (1 + float((gr.abs() * d.abs()).sum()) ** 0.5 + abs(want))


GATED_CASES = [
    # batch, seqlen, dim, group_size, dtype, z, before, elements before / after z in its row
    (1, 1, 1, 1, F32, True, False, 0, 0), (2, 3, 24, 8, BF, True, True, 8, 16),
    (2, 5, 21, 7, BF, True, False, 1, 2), (1, 33, 100, 100, F32, True, True, 3, 0),
    (2, 37, 640, 128, BF, False, False, 0, 0), (1, 8, 5120, 5120, BF, True, False, 0, 336),
    (3, 211, 5120, 640, BF, True, False, 0, 336), (1, 150, 1024, 256, F32, True, True, 4, 4),
    (1, 3, 8200, 8200, F32, True, False, 0, 0), (1, 2, 16384, 16384, BF, True, True, 0, 0),
    (2, 1000, 16, 8, F32, True, False, 0, 8),
]


def _gated_inputs(B, L, dim, gs, dt, has_z, before, pre, post):
    g = torch.Generator().manual_seed(B * 7 + L + dim)
    y = (torch.randn(B, L, dim, generator=g) * 2).to(dt)
    src = torch.randn(B, L, pre + dim + post, generator=g).to(dt)
    w = torch.randn(dim, generator=g) * 0.3 + 1
    dout = torch.randn(B, L, dim, generator=g).to(dt)
    return y, src, w, dout


@pytest.mark.parametrize("case", GATED_CASES, ids=str)
def test_gated_rmsnorm(case):
    import selective_state_space_05_gb300 as ssd
    B, L, dim, gs, dt, has_z, before, pre, post = case
    y, src, w, dout = _gated_inputs(*case)
    cy, csrc, cw, cdo = _cuda(y, src, w, dout)
    z = src[:, :, pre:pre + dim] if has_z else None
    cz = csrc[:, :, pre:pre + dim] if has_z else None
    kw = dict(group_size=gs, eps=1e-5, norm_before_gate=before)
    out = ssd.gated_rmsnorm_fwd(cy, cz, cw, **kw)
    Y, Z, W = bt.leaf(y), bt.leaf(z), bt.leaf(w)
    ref = bt.gated_rmsnorm(Y, Z, W, gs, 1e-5, before)
    bt.assert_within(out, ref.detach(), ref.detach().abs(), OPS, "out")
    # the gradient written into a slice of a larger one, whose rest stays
    buf = torch.full_like(csrc, 7.0)
    dz = buf[:, :, pre:pre + dim] if has_z else None
    got = ssd.gated_rmsnorm_bwd(cdo, cy, cz, cw, dz=dz, **kw)
    leaves = [t for t in (Y, Z, W) if t is not None]
    grads = dict(zip([n for n, t in (("dy", Y), ("dz", Z), ("dweight", W)) if t is not None],
                     torch.autograd.grad(ref, leaves, dout.double())))
    # magnitudes of the formulas' terms
    with torch.no_grad():
        e = bt.silu(Z).abs() if has_z else torch.ones_like(Y)
        de = bt.dsilu_mag(Z) if has_z else torch.zeros_like(Y)
        u = (Y.abs() if before else Y.abs() * e)
        ug = u.unflatten(-1, (-1, gs))
        rms = (ug.square().mean(-1, keepdim=True) + 1e-5).sqrt().expand_as(ug).flatten(-2)
        g = (dout.double() * W).abs() * (e if before else 1)
        n = u / rms
        gn = (g * n).unflatten(-1, (-1, gs)).mean(-1, keepdim=True).expand_as(ug).flatten(-2)
        du = (g + n * gn) / rms
        mags = dict(dy=du if before else du * e,
                    dz=(dout.double() * W).abs() * n * de if before else du * Y.abs() * de,
                    dweight=(dout.double().abs() * n * (e if before else 1)).sum((0, 1)))
    for k, v in grads.items():
        bt.assert_within(got[k], v, mags[k], _sum_ops(B * L) if k == "dweight" else OPS, k)
    if has_z:
        assert (buf[:, :, :pre] == 7).all() and (buf[:, :, pre + dim:] == 7).all()
    else:
        assert got["dz"] is None


def test_gated_rmsnorm_matches_group_rmsnorm():
    """Without a gate it is the framework's in-place group norm."""
    import selective_state_space_05_gb300 as ssd
    y = torch.randn(2, 9, 512, device="cuda")
    w = torch.randn(512, device="cuda")
    a = ssd.gated_rmsnorm_fwd(y, None, w, group_size=128)
    b = ssd.group_rmsnorm_(y.clone(), w, group_size=128)
    assert (a - b).abs().max() <= 1e-5 * b.abs().max()


def test_gated_rmsnorm_autograd_shapes_and_streams():
    import selective_state_space_05_gb300 as ssd
    proj = torch.randn(2, 7, 3 * 64, device="cuda").requires_grad_(True)
    y = torch.randn(2, 7, 64, device="cuda").requires_grad_(True)
    w = torch.ones(64, device="cuda").requires_grad_(True)
    out = ssd.gated_rmsnorm(y, proj[..., 64:128], w, group_size=32, norm_before_gate=True)
    out.square().sum().backward()
    Y, Z, W = bt.leaf(y), bt.leaf(proj[..., 64:128]), bt.leaf(w)
    bt.gated_rmsnorm(Y, Z, W, 32, 1e-5, True).square().sum().backward()
    for a, b in ((y.grad, Y.grad), (proj.grad[..., 64:128], Z.grad), (w.grad, W.grad)):
        assert (a.double().cpu() - b).abs().max() <= 1e-5 * b.abs().max()
    assert (proj.grad[..., :64] == 0).all() and (proj.grad[..., 128:] == 0).all()
    # another stream, workspaces allocated there
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ssd.gated_rmsnorm_bwd(torch.ones(2, 7, 64, device="cuda"), y.detach(), None, w.detach(),
                                stream=side)
    side.synchronize()
    ref = ssd.gated_rmsnorm_bwd(torch.ones(2, 7, 64, device="cuda"), y.detach(), None, w.detach())
    assert torch.equal(got["dweight"], ref["dweight"])
    # an empty batch is refused, as by the other calls of the library
    with pytest.raises(ssd._lib.SSDError):
        ssd.gated_rmsnorm_fwd(y.detach()[:0], None, w.detach())


def test_norms_in_a_graph():
    """The explicit calls captured and replayed give the eager bits."""
    import selective_state_space_05_gb300 as ssd
    x, r, w = (torch.randn(40, 256, device="cuda"), torch.randn(40, 256, device="cuda"),
               torch.randn(256, device="cuda"))

    def step():
        y, ro = ssd.add_rmsnorm_fwd(x, r, w)
        return ssd.add_rmsnorm_bwd(y, ro, ro, w)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for k in ("dx", "dresidual", "dweight"):
        assert torch.equal(want[k], got[k])
