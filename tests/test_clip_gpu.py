"""Gradient norm and clipping on the GPU against 64 bits."""
import math

import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
U = 2.0 ** -24


def _ref_norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def _sets():
    g = torch.Generator().manual_seed(11)

    def r(*s, dt=F32):
        return torch.randn(*s, generator=g).to(dt)
    yield "one element", [r(1)]
    yield "empty among others", [r(0), r(5), r(0, 3), r(7, 3, dt=BF)]
    yield "many small", [r(i % 37 + 1, dt=BF if i % 3 else F32) for i in range(900)]
    yield "chunk borders", [r(16384), r(16385, dt=BF), r(32767), r(3, 5461)]
    yield "one long", [r(3_000_001, dt=BF)]
    flat = r(2 * 10007)
    yield "unaligned views", [flat[1:10004], flat[10004:10007], flat[10007:]]
    yield "transposed", [r(64, 48).t(), r(8, 4, 6).permute(2, 0, 1)]


SETS = dict(_sets())


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("factor", [0.25, 2.0])
@pytest.mark.parametrize("to", ["in", "same", "f32", "bf16"])
def test_clip(name, factor, to):
    import selective_state_space_05_gb300 as ssd
    ts = SETS[name]
    dev = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)
           if name == "transposed" else t.cuda() for t in ts]
    if name == "unaligned views":
        flat = torch.cat([t.flatten() for t in ts])
        base = torch.empty(flat.numel() + 1, device="cuda")
        base[1:] = flat.cuda()
        dev = list(base[1:].split([t.numel() for t in ts]))
    ref = _ref_norm(ts)
    limit = factor * ref
    out = None
    if to != "in":
        out = [torch.empty_like(d, dtype={"same": d.dtype, "f32": F32, "bf16": BF}[to])
               for d in dev]
    norm = ssd.clip_grads(dev, limit, out=out)
    assert norm.dtype == F32 and norm.dim() == 0
    # squares summed in fp32 over at most 64 values of a thread, then in double
    assert abs(float(norm) - ref) <= 66 * U * ref
    coef = min(1.0, limit / (ref + 1e-6))
    for t, d, o in zip(ts, dev, out or dev):
        # the norm's error, the factor's and the product's rounding
        bt.assert_within(o, t.double() * coef, (t.double() * coef).abs(), 70, name)
        if to != "in":
            assert torch.equal(d.cpu(), t)
        elif factor > 1:
            assert torch.equal(o.cpu(), t)
    assert abs(float(ssd.grad_norm([t.cuda() for t in ts])) - ref) <= 66 * U * ref


@pytest.mark.parametrize("size", [1e-30, 1e-19, 1e20, 1e36])
def test_range(size):
    """Squares outside fp32's range."""
    import selective_state_space_05_gb300 as ssd
    t = torch.randn(1000, generator=torch.Generator().manual_seed(1)) * size
    t[::7] = 0
    ref = _ref_norm([t])
    assert abs(float(ssd.grad_norm(t.cuda())) - ref) <= 66 * U * ref


def test_not_finite():
    import selective_state_space_05_gb300 as ssd
    a, b = torch.ones(100, device="cuda"), torch.ones(3, device="cuda", dtype=BF)
    a[50] = float("inf")
    norm = ssd.clip_grads([a, b], 1.0)
    assert float(norm) == math.inf
    assert torch.isnan(a[50]) and a[49] == 0 and (b == 0).all()
    a = torch.ones(100, device="cuda")
    a[3] = float("nan")
    norm = ssd.clip_grads([a], 1.0)
    assert math.isnan(float(norm)) and torch.isnan(a).all()


def test_repeats_are_equal_and_graphs_work():
    import selective_state_space_05_gb300 as ssd
    g = [torch.randn(100_003, device="cuda"), torch.randn(64, 33, device="cuda").to(BF)]
    o = [torch.empty_like(t) for t in g]
    first = ssd.clip_grads(g, 1.0, out=o)
    want = [t.clone() for t in o]
    for _ in range(3):
        assert torch.equal(ssd.clip_grads(g, 1.0, out=o), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = ssd.clip_grads(g, 1.0, out=o)
    for t in o:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(o, want))


def test_refusals():
    import selective_state_space_05_gb300 as ssd
    a = torch.ones(4, 4, device="cuda")
    for bad in ([], [None], [a.half()], [a.cpu()], [a[:, :2]]):
        with pytest.raises(ValueError):
            ssd.clip_grads(bad, 1.0)
    with pytest.raises(ValueError, match="twice"):
        ssd.clip_grads([a, a], 1.0)
    with pytest.raises(ValueError, match="out"):
        ssd.clip_grads([a], 1.0, out=[a, a])
    with pytest.raises(ValueError, match="match"):
        ssd.clip_grads([a], 1.0, out=[torch.ones(4, 5, device="cuda")])
    with pytest.raises(ssd._lib.SSDError):
        ssd.clip_grads([a], -1.0)
    assert (a == 1).all()
