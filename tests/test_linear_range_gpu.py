"""fp32 projections of operands at the ends of the type's range: infinities,
NaN and the largest finite values give the 64-bit product's infinities, NaN and
finite values, whichever kernel the number of rows selects."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32 = torch.float32
INF, NAN = float("inf"), float("nan")
MAX = torch.finfo(F32).max

# rows on both sides of the few-rows border, K on and off the 16-byte grid, and
# sums of several runs
SHAPES = [(20, 200, 136), (300, 200, 136), (20, 201, 136), (300, 201, 133), (140, 1030, 40)]


def dot(a, b):
    """sum_k a[m,k] b[n,k] in 64 bits, term by term."""
    out = torch.empty(a.shape[0], b.shape[0], dtype=torch.float64)
    for m in range(a.shape[0]):
        out[m] = (a[m].double() * b.double()).sum(-1)
    return out


def _ops(K):
    return 8 * (K // 16 + 1) + 64


def check(got, ref, mag, ops, what):
    """NaN and infinities where ref has them; finite values within the bound."""
    g = got.detach().double().cpu()
    inf = torch.isinf(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaNs differ"
    assert torch.equal(torch.where(inf, g, 0.0), torch.where(inf, ref, 0.0)), f"{what}: infinities"
    rest = ~inf & ~torch.isnan(ref)
    zero = torch.zeros_like(ref)
    bt.assert_within(torch.where(rest, g, zero).to(got.dtype), torch.where(rest, ref, zero),
                     torch.where(rest, mag, zero), ops, what)


def operands(M, K, N, seed=0):
    g = torch.Generator().manual_seed(M + K + N + seed)
    x = torch.randn(M, K, generator=g)
    w = torch.randn(N, K, generator=g) * K ** -0.5
    w.clamp_(-0.9, 0.9)
    return x, w


def plant(x, w):
    x[:, 8] *= 1e-3                    # against w's largest values
    x[7, 5], x[9, 3], x[13, 2] = INF, -INF, NAN
    x[11, 0], x[11, 1] = INF, -INF
    x[15, 4], x[16, 6] = -MAX, MAX
    w[20, 6], w[21, 7] = INF, -INF
    w[22, 8], w[24, 8] = -MAX, 0.999 * MAX
    w[23, 5] = 0.0                     # infinity times zero


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("form", ["plain", "bias silu", "residual", "residual in place"])
def test_forward(shape, form):
    import selective_state_space_05_gb300 as ssd
    x, w = operands(*shape)
    plant(x, w)
    M, K, N = shape
    b = torch.randn(N, generator=torch.Generator().manual_seed(1)) if "bias" in form else None
    r = torch.randn(M, N, generator=torch.Generator().manual_seed(2)) if "res" in form else None
    act = "silu" if "silu" in form else None
    cr = None if r is None else r.cuda()
    got = ssd.linear_fwd(x.cuda(), w.cuda(), None if b is None else b.cuda(), activation=act,
                         residual=cr, out=cr if "place" in form else None, save_pre=act is not None)
    out, pre = got if act else (got, None)
    ssd.scan_status()
    ref, mag = dot(x, w), dot(x.abs(), w.abs())
    if b is not None:
        ref, mag = ref + b.double(), mag + b.double().abs()
    if act:
        check(pre, ref, mag, _ops(K), "pre")
        ref, mag = bt.silu(ref), 1.13 * mag
    if r is not None:
        ref, mag = ref + r.double(), mag + r.double().abs()
    check(out, ref, mag, _ops(K), "out")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("where", ["x", "w", "dout", "all"])
@pytest.mark.parametrize("act", [None, "silu"])
def test_backward(shape, where, act):
    import selective_state_space_05_gb300 as ssd
    M, K, N = shape
    x, w = operands(*shape)
    g = torch.Generator().manual_seed(3)
    do = torch.randn(M, N, generator=g)
    pre = torch.randn(M, N, generator=g)
    x2, w2 = x.clone(), w.clone()
    plant(x2, w2)
    if where in ("x", "all"):
        x = x2
        do[:, 1] *= 1e-3
        do[15] *= 1e-2
        do[16] *= 1e-2
    if where in ("w", "all"):
        w = w2
        do[:, 22] *= 1e-3
        do[:, 24] *= 1e-3
    if where in ("dout", "all"):
        do[4, 9], do[6, 30], do[8, 31], do[10, 3] = INF, -INF, NAN, -0.05 * MAX
    got = ssd.linear_bwd(do.cuda(), x.cuda(), w.cuda(), activation=act,
                         pre=pre.cuda() if act else None, need_dbias=True)
    ssd.scan_status()
    d = do.double()
    if act:
        p = pre.double()
        s = 1 / (1 + torch.exp(-p))
        d = d * s * (1 + p * (1 - s))
    # silu' has its roundings relative to its terms, which cancel near -1.28
    a = do.double().abs() * bt.dsilu_mag(p) if act else d.abs()
    check(got["dx"], dot(d, w.t()), dot(a, w.t().abs()), _ops(N), "dx")
    check(got["dweight"], dot(d.t(), x.t()), dot(a.t(), x.t().abs()), _ops(M), "dweight")
    check(got["dbias"], d.sum(0), a.sum(0), M + 64, "dbias")


def test_largest_values_alone():
    """Finite operands give finite values: the mask of the type's lowest value."""
    import selective_state_space_05_gb300 as ssd
    for M in (16, 400):
        x = torch.full((M, 256), -MAX)
        x[:, 1:] = 0
        w = torch.full((64, 256), 1.0)
        w[1::2] = 1e-5
        out = ssd.linear_fwd(x.cuda(), w.cuda()).cpu()
        assert (out[:, 0::2] == -MAX).all()
        want = -MAX * float(torch.tensor(1e-5))
        assert ((out[:, 1::2].double() - want).abs() <= 8 * bt.U32 * abs(want)).all()


def test_nothing_but_nan():
    """A step that has diverged stays as fast as a launch or two."""
    import selective_state_space_05_gb300 as ssd
    x = torch.full((700, 520), NAN, device="cuda")
    w = torch.randn(300, 520, device="cuda")
    assert torch.isnan(ssd.linear_fwd(x, w)).all()
    w[7, 519] = INF
    g = ssd.linear_bwd(torch.full((700, 300), -INF, device="cuda"), x.nan_to_num(1.0), w)
    assert torch.isinf(g["dweight"]).all() and not torch.isfinite(g["dx"]).any()


def test_a_few_places_of_a_large_product():
    """Their rows and columns only: every other result keeps the bits it has
    without them."""
    import selective_state_space_05_gb300 as ssd
    M, K, N = 2000, 2100, 1500
    g = torch.Generator("cuda").manual_seed(9)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, w, do = r(M, K), r(N, K) * K ** -0.5, r(M, N)
    places = {"x": (x, [(0, 0), (777, 1024), (1999, 2099)]), "w": (w, [(3, 5), (1499, 2099)]),
              "do": (do, [(1, 1023), (1024, 7), (1998, 1499)])}
    for t, at in places.values():
        for i, j in at:
            t[i, j] = 0.0

    def step():
        b = ssd.linear_bwd(do, x, w)
        return ssd.linear_fwd(x, w), b["dx"], b["dweight"]

    clean = step()
    for n, (t, at) in enumerate(places.values()):
        for k, (i, j) in enumerate(at):
            t[i, j] = (INF, -INF, NAN)[(n + k) % 3]
    got = step()
    rows = {k: [i for i, _ in at] for k, (_, at) in places.items()}
    cols = {k: [j for _, j in at] for k, (_, at) in places.items()}
    # the three products, which rows and columns of each are concerned, and the terms
    for name, a, b, out, was, ar, bc in (
            ("out", x, w, got[0], clean[0], rows["x"], rows["w"]),
            ("dx", do, w.t(), got[1], clean[1], rows["do"], cols["w"]),
            ("dweight", do.t(), x.t(), got[2], clean[2], cols["do"], cols["x"])):
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        hit[ar] = True
        hit[:, bc] = True
        assert torch.equal(out[~hit], was[~hit]), name
        for i in ar:
            ref = (a[i].double() * b.double()).sum(-1).float()
            assert torch.equal(torch.isnan(out[i]), torch.isnan(ref)), (name, i)
            assert torch.equal(out[i].nan_to_num(7.0), ref.nan_to_num(7.0)), (name, i)
        for j in bc:
            ref = (a.double() * b[j].double()).sum(-1).float()
            assert torch.equal(torch.isnan(out[:, j]), torch.isnan(ref)), (name, j)
            assert torch.equal(out[:, j].nan_to_num(7.0), ref.nan_to_num(7.0)), (name, j)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rt", [None, F32])
def test_bf16(shape, rt):
    """bf16 operands go to the tensor cores as they are."""
    import selective_state_space_05_gb300 as ssd
    bf = torch.bfloat16
    M, K, N = shape
    x, w = operands(*shape)
    plant(x, w)
    big = torch.finfo(bf).max

    def to_bf16(t):   # the largest fp32 values would round to infinities
        return torch.where(torch.isfinite(t), t.clamp(-big, big), t).to(bf)
    x, w = to_bf16(x), to_bf16(w)
    r = torch.randn(M, N, generator=torch.Generator().manual_seed(2)) if rt else None
    out = ssd.linear_fwd(x.cuda(), w.cuda(), residual=None if r is None else r.cuda())
    ref, mag = dot(x, w), dot(x.abs(), w.abs())
    if r is not None:
        ref, mag = ref + r.double(), mag + r.double().abs()
    check(out, ref, mag, _ops(K), "out")
    do = torch.randn(M, N, generator=torch.Generator().manual_seed(3))
    do[:, 1] *= 1e-3
    do[15] *= 1e-2
    do[16] *= 1e-2
    do[:, 22] *= 1e-3
    do[:, 24] *= 1e-3
    do[4, 9], do[6, 30], do[8, 31], do[10, 3] = INF, -INF, NAN, -0.05 * MAX
    do = do.to(bf)
    got = ssd.linear_bwd(do.cuda(), x.cuda(), w.cuda(), need_dbias=True)
    ssd.scan_status()
    d, a = do.double(), do.double().abs()
    check(got["dx"], dot(d, w.t()), dot(a, w.t().abs()), _ops(N), "dx")
    check(got["dweight"], dot(d.t(), x.t()), dot(a.t(), x.t().abs()), _ops(M), "dweight")
    check(got["dbias"], d.sum(0), a.sum(0), M + 64, "dbias")
