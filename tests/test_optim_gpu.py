"""AdamW over many tensors on the GPU: against its definition in 64 bits, and the
8-bit moments against the same arithmetic in torch on the CPU, code by code."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U32 = 2.0 ** -24
SIZES = [(1,), (7,), (8,), (0,), (255,), (256,), (257,), (3, 85), (64, 130), (8191,), (8192,),
         (8193,), (20000,)]


@pytest.fixture(scope="module")
def ssd():
    import selective_state_space_05_gb300 as m
    return m


def make(shapes, pdt, gdt, bits, master, seed=0, offset=0):
    """Parameters, gradients and a state with moments, cut from buffers that
    start `offset` elements in."""
    gen = torch.Generator().manual_seed(seed)
    n = sum(math.prod(s) for s in shapes) + offset

    def cut(flat):
        got, at = [], offset
        for s in shapes:
            k = math.prod(s)
            got.append(flat[at:at + k].view(s))
            at += k
        return got

    w = torch.randn(n, generator=gen) * 0.05
    g = (torch.randn(n, generator=gen) * 1e-3).to(gdt)
    p = w.to(pdt)
    state = dict(master=[t if pdt is BF else None for t in cut(w.cuda())] if master else None)
    if bits == 32:
        state.update(exp_avg=cut((torch.randn(n, generator=gen) * 3e-4).cuda()),
                     exp_avg_sq=cut((torch.rand(n, generator=gen) * 2e-6).cuda()))
    else:
        state.update(
            exp_avg=cut(torch.randint(-127, 128, (n,), generator=gen).to(torch.int8).cuda()),
            exp_avg_sq=cut(torch.randint(0, 256, (n,), generator=gen).to(torch.uint8).cuda()),
            exp_avg_scale=[(torch.rand(-(-math.prod(s) // 256), generator=gen) * 1e-3).cuda()
                           for s in shapes],
            exp_avg_sq_scale=[(torch.rand(-(-math.prod(s) // 256), generator=gen) * 3e-6).cuda()
                              for s in shapes])
    return cut(p.cuda()), cut(g.cuda()), state


def values(state, i):
    """Moments of tensor i in fp32, on the CPU."""
    m, v = state["exp_avg"][i].cpu().flatten(), state["exp_avg_sq"][i].cpu().flatten()
    if m.dtype is F32:
        return m, v
    blk = torch.arange(m.numel()) // 256
    t = m.float() * torch.tensor(1.0 / 127.0)
    u = v.float() * torch.tensor(1.0 / 255.0)
    u = u * u
    return ((t * t.abs()) * state["exp_avg_scale"][i].cpu()[blk],
            (u * u) * state["exp_avg_sq_scale"][i].cpu()[blk])


def definition(p, g, m, v, step, lr, betas, eps, decay, coef):
    p, g, m, v = (t.double().cpu().flatten() for t in (p, g, m, v))
    g = g * coef
    mag = betas[0] * m.abs() + (1 - betas[0]) * g.abs()
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    over = lr / (1 - betas[0] ** step) / ((v / (1 - betas[1] ** step)).sqrt() + eps)
    return p - lr * decay * p - over * m, m, v, mag, over


def within(got, ref, ops, what, extra=0.0):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double().cpu().flatten() - ref).abs()
    bound = half * ref.abs() * 1.01 + ops * U32 * ref.abs() + extra + 2.0 ** -126
    assert (err <= bound).all(), f"{what}: {float((err / bound).max()):.3g} times its bound"


HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def reference(p, g, state, step, coef=1.0, hyper=HYPER):
    """definition() of each tensor, before the step."""
    res = []
    for i in range(len(p)):
        w = p[i]
        if state.get("master") is not None and state["master"][i] is not None:
            w = state["master"][i]
        m, v = values(state, i)
        res.append(definition(w, g[i], m, v, step, hyper["lr"], hyper["betas"], hyper["eps"],
                              hyper["weight_decay"], coef))
    return res


def compare(p, state, want):
    for i, (rp, rm, rv, mag, over) in enumerate(want):
        # m is a sum of two terms, `mag` their sizes' sum: the constants' and the
        # operations' roundings (two a term, with the clipping's three, and the sum's) are
        # 8 of mag.  The update adds six fp32 operations, v's six roundings halved
        # by the root, and the approximate root and division, 2^-21 (8 roundings)
        # each: 8 + 6 + 3 + 16 < 36 of over * mag; and p's factor rounds once
        err = 8 * U32 * mag
        extra = 36 * U32 * over * mag + 2 * U32 * rp.abs()
        if state.get("master") is not None and state["master"][i] is not None:
            within(state["master"][i], rp, 1, f"master {i}", extra)
        within(p[i], rp, 1, f"param {i}", extra)
        if state["exp_avg"][i].dtype is F32:
            within(state["exp_avg"][i], rm, 0, f"m {i}", err)
            # v's terms are not negative; the clipping counts twice in g'^2
            within(state["exp_avg_sq"][i], rv, 12, f"v {i}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt,master", [(F32, F32, False), (BF, BF, True), (BF, F32, True),
                                            (BF, BF, False), (F32, BF, False), (F32, F32, True)])
def test_against_the_definition(ssd, bits, pdt, gdt, master):
    for offset in (0, 1, 3):
        p, g, state = make(SIZES, pdt, gdt, bits, master, seed=offset, offset=offset)
        norm = ssd.grad_norm(g)
        for step, clip in ((1, None), (1000, 0.3)):
            coef = 1.0 if clip is None else min(1.0, clip * float(norm) / (float(norm) + 1e-6))
            kw = {} if clip is None else dict(grad_norm=norm, max_norm=clip * float(norm))
            want = reference(p, g, state, step, coef)
            before = [t.clone() for t in g]
            ssd.adamw_step(p, g, state, step=step, seed=5, **HYPER, **kw)
            compare(p, state, want)
            assert all(torch.equal(a, b) for a, b in zip(before, g))


def mix(h):
    low = 0xFFFFFFFF
    h = ((h ^ (h >> 16)) * 0x7FEB352D) & low
    h = ((h ^ (h >> 15)) * 0x846CA68B) & low
    return h ^ (h >> 16)


def encode(x, u, top, power):
    """Codes and scales of x >= 0, one operation a line of the kernel's."""
    n = x.numel()
    full = torch.zeros(-(-n // 256) * 256)
    full[:n] = x
    big = full.view(-1, 256).amax(1)
    r = torch.where(x > 0, x / big[torch.arange(n) // 256], torch.zeros(n))
    y = torch.sqrt(r) if power == 2 else torch.sqrt(torch.sqrt(r))
    c = torch.clamp(torch.floor(y * top), max=top - 1)

    def unit(c):
        t = c * torch.tensor(1.0 / top)
        return t * t if power == 2 else (t * t) * (t * t)
    lo, hi = unit(c), unit(c + 1)
    return c + (u < (r - lo) / (hi - lo)).float(), big


@pytest.mark.parametrize("seed,step", [(0, 1), (12345, 77)])
def test_codes_bit_by_bit(ssd, seed, step):
    p, g, state = make(SIZES, BF, F32, 8, True, seed=3)
    want = []
    for i in range(len(p)):
        m, v = values(state, i)
        b1, b2 = HYPER["betas"]
        gi = g[i].cpu().flatten()
        m = m * b1 + gi * (1.0 - b1)
        v = v * b2 + (gi * gi) * (1.0 - b2)
        low = 0xFFFFFFFF
        key = mix((mix((mix(torch.tensor(seed)) + step) & low) + i) & low)
        h = mix((key + torch.arange(m.numel())) & low)
        cm, ms = encode(m.abs(), ((h >> 16).float() + 0.5) * 2.0 ** -16, 127.0, 2)
        cv, vs = encode(v, ((h & 0xFFFF).float() + 0.5) * 2.0 ** -16, 255.0, 4)
        want.append((cm * torch.sign(m), ms, torch.where(v > 0, cv.clamp(min=1), cv), vs))
    ssd.adamw_step(p, g, state, step=step, seed=seed, **HYPER)
    for i, (cm, ms, cv, vs) in enumerate(want):
        assert torch.equal(state["exp_avg"][i].cpu().flatten().float(), cm), i
        assert torch.equal(state["exp_avg_sq"][i].cpu().flatten().float(), cv), i
        assert torch.equal(state["exp_avg_scale"][i].cpu(), ms)
        assert torch.equal(state["exp_avg_sq_scale"][i].cpu(), vs)
    out = ssd.adamw_moments(state)
    for i in range(len(p)):
        m, v = values(state, i)
        assert torch.equal(out[0][i].cpu().flatten(), m) and out[0][i].shape == p[i].shape
        assert torch.equal(out[1][i].cpu().flatten(), v)


def test_codes_at_their_edges(ssd):
    """A first step's codes, bit by bit, for gradients of all sizes that fp32 squares
    hold and past them, for values that are a code's own and next to it, for blocks of
    zeros, and for four million values in all."""
    gen = torch.Generator().manual_seed(9)
    blocks = 16384
    n = blocks * 256 - 100
    g = torch.randn(blocks, 256, generator=gen)
    g *= 10.0 ** (torch.rand(blocks, 1, generator=gen) * 38 - 21)     # 1e-21 to 1e17
    m_code = torch.randint(0, 128, (blocks, 256), generator=gen).float() / 127
    v_code = torch.randint(0, 256, (blocks, 256), generator=gen).float() / 255
    near = 1 + (torch.randint(-2, 3, (blocks, 256), generator=gen)).float() * 2.0 ** -23
    size = 10.0 ** (torch.rand(blocks, 1, generator=gen) * 8 - 6)
    kind = torch.arange(blocks)[:, None] % 4
    g = torch.where(kind == 1, m_code ** 2 * near * size, g)
    g = torch.where(kind == 2, -v_code ** 2 * near * size, g)
    g[3::64] = 0.0
    g = g.flatten()[:n].contiguous()
    m, v = g * (1.0 - 0.9) + 0.0, (g * g) * (1.0 - 0.999)
    low = 0xFFFFFFFF
    key = mix((mix((mix(torch.tensor(21)) + 1) & low) + 0) & low)
    h = mix((key + torch.arange(n)) & low)
    cm, ms = encode(m.abs(), ((h >> 16).float() + 0.5) * 2.0 ** -16, 127.0, 2)
    cv, vs = encode(v, ((h & 0xFFFF).float() + 0.5) * 2.0 ** -16, 255.0, 4)
    p = [torch.zeros(n, device="cuda")]
    state = ssd.adamw_state(p, bits=8)
    ssd.adamw_step(p, [g.cuda()], state, step=1, lr=1e-3, betas=(0.9, 0.999), seed=21)
    assert torch.equal(state["exp_avg_scale"][0].cpu(), ms)
    assert torch.equal(state["exp_avg_sq_scale"][0].cpu(), vs)
    assert torch.equal(state["exp_avg"][0].cpu().float(), cm * torch.sign(m))
    assert torch.equal(state["exp_avg_sq"][0].cpu().float(), torch.where(v > 0, cv.clamp(min=1), cv))


def test_rounded_averages_keep_moving(ssd):
    """Each new moment's steps are below half a code's, yet the averages arrive:
    with gradients of one size v tends to their square as 1 - beta2^t.  The mean
    over 65536 elements of independent roundings is off by much less than the
    bound: each rounding moves a value by at most a code's step (4/160 of it
    here) and forgets with beta2, so the mean's deviation is below
    (4/160) / sqrt(2 (1 - beta2) 65536) = 0.22 %; the bound is 8 of them."""
    n = 65536
    p = [torch.zeros(n, device="cuda")]
    g = [torch.full((n,), 1e-3, device="cuda")]
    g[0][::256] = 2e-3        # each block's largest: the others' codes are near 180
    state = ssd.adamw_state(p, bits=8)
    for t in range(1, 1501):
        ssd.adamw_step(p, g, state, step=t, lr=0.0, betas=(0.9, 0.999), seed=9)
    m, v = ssd.adamw_moments(state)
    rest = torch.arange(n, device="cuda") % 256 != 0
    want = 1e-6 * (1 - 0.999 ** 1500)
    assert abs(float(v[0][rest].mean()) / want - 1) < 0.018
    assert abs(float(m[0][rest].mean()) / 1e-3 - 1) < 0.005


def test_missing_gradients_and_numbers(ssd):
    """A gradient None leaves its parameter and moments, and the others' roundings
    as they would be."""
    p, g, state = make(SIZES, F32, F32, 8, False, seed=4)
    q, h, other = make(SIZES, F32, F32, 8, False, seed=4)
    none = [None if i in (2, 7, 9) else t for i, t in enumerate(g)]
    ssd.adamw_step(p, none, state, step=3, **HYPER)
    kept = [(q[i].clone(), other["exp_avg"][i].clone()) for i in range(len(q))]
    ssd.adamw_step(q, h, other, step=3, **HYPER)
    for i in range(len(p)):
        if none[i] is None:
            assert torch.equal(p[i], kept[i][0]) and torch.equal(state["exp_avg"][i], kept[i][1])
        else:
            assert torch.equal(p[i], q[i])
            for n in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
                assert torch.equal(state[n][i], other[n][i]), n
    ssd.adamw_step([], [], ssd.adamw_state([]), step=1, lr=1e-3)
    ssd.adamw_step(p, [None] * len(p), state, step=1, lr=1e-3)
    a, b = torch.ones(3, device="cuda"), torch.ones(4, device="cuda")
    ssd.adamw_step([a, b], [None, b.clone()], ssd.adamw_state([a, b]), step=1, lr=1e-3)
    assert (a._version, b._version) == (0, 1)
    # one tensor instead of lists of one
    a, b = q[4].clone(), h[4]
    ssd.adamw_step(a, b, ssd.adamw_state(a), step=1, lr=1e-2, weight_decay=0.0)
    assert (a - q[4] + 1e-2 * torch.sign(b)).abs().max() <= 1e-4


def test_device_step_and_rate_in_a_graph(ssd):
    """A captured step reads the step's number, the rate and the norm anew."""
    for bits in (32, 8):
        p, g, state = make(SIZES, BF, BF, bits, True, seed=6)
        q, h, other = make(SIZES, BF, BF, bits, True, seed=6)
        step = torch.zeros((), dtype=torch.int64, device="cuda")
        lr = torch.zeros((), device="cuda")
        kw = dict(betas=(0.9, 0.95), weight_decay=0.02, seed=2)

        def one():
            step.add_(1)
            norm = ssd.grad_norm(g)
            ssd.adamw_step(p, g, state, step=step, lr=lr, grad_norm=norm, max_norm=0.05, **kw)
        one()                        # with a rate of 0, on both sides
        ssd.adamw_step(q, h, other, step=1, lr=0.0, grad_norm=ssd.grad_norm(h), max_norm=0.05, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one()
        for t in range(2, 6):
            lr.fill_(2.0 ** -t)
            for a, b in zip(g, h):
                a.mul_(1.5)
                b.copy_(a)
            graph.replay()
            ssd.adamw_step(q, h, other, step=t, lr=2.0 ** -t, grad_norm=ssd.grad_norm(h),
                           max_norm=0.05, **kw)
        for i in range(len(p)):
            assert torch.equal(p[i], q[i]), (bits, i)
            assert torch.equal(state["master"][i], other["master"][i])
            assert torch.equal(state["exp_avg"][i], other["exp_avg"][i])


def test_many_tensors_strides_and_streams(ssd):
    """More tensors than a launch takes, dense tensors of other strides, a side
    stream."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    p = [torch.randn(3 + i % 5, 7, generator=gen, device="cuda") for i in range(800)]
    p[5] = torch.randn(6, 4, 5, generator=gen, device="cuda").permute(2, 0, 1)
    g = [torch.randn_like(t) for t in p]
    assert not g[5].is_contiguous()
    state = ssd.adamw_state(p)
    want = reference(p, g, state, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ssd.adamw_step(p, g, state, step=2, stream=side, **HYPER)
    side.synchronize()
    compare(p, state, want)
    assert p[3]._version == 1 and state["exp_avg"][3]._version == 1 and g[3]._version == 0
    with pytest.raises(ValueError, match="strides"):
        ssd.adamw_step(p, [t.contiguous() for t in g], state, step=2, **HYPER)


def test_values_that_are_not_finite(ssd):
    for bits in (32, 8):
        p, g, state = make([(1000,)], F32, F32, bits, False, seed=8)
        q, h, other = make([(1000,)], F32, F32, bits, False, seed=8)
        g[0][300] = float("nan")
        g[0][310] = float("inf")
        ssd.adamw_step(p, g, state, step=1, **HYPER)
        ssd.adamw_step(q, h, other, step=1, **HYPER)
        bad = torch.zeros(1000, dtype=torch.bool, device="cuda")
        bad[[300, 310]] = True
        assert torch.equal(p[0][~bad], q[0][~bad])
        assert torch.isnan(p[0][300])
        m, _ = ssd.adamw_moments(state)
        n, _ = ssd.adamw_moments(other)
        far = torch.arange(1000, device="cuda") // 256 != 1 if bits == 8 else ~bad
        assert torch.equal(m[0][far], n[0][far]) and not torch.isfinite(m[0][300])
    # a norm that is not a number makes all so; an infinite one leaves no gradient
    p, g, state = make([(300,)], F32, F32, 32, False, seed=9)
    q = p[0].clone()
    m = state["exp_avg"][0].clone()
    inf = torch.tensor(float("inf"), device="cuda")
    ssd.adamw_step(p, g, state, step=1, grad_norm=inf, max_norm=1.0, lr=0.0, weight_decay=0.0)
    assert torch.equal(p[0], q) and torch.equal(state["exp_avg"][0], m * 0.9)
    ssd.adamw_step(p, g, state, step=1, grad_norm=inf - inf, max_norm=1.0, lr=0.1)
    assert torch.isnan(p[0]).all()


def test_zero_blocks(ssd):
    """Blocks whose moments are all 0 stay so, and a v above 0 keeps a code."""
    p = [torch.ones(600, device="cuda")]
    g = [torch.zeros(600, device="cuda")]
    state = ssd.adamw_state(p, bits=8)
    ssd.adamw_step(p, g, state, step=1, lr=0.1, weight_decay=0.0)
    assert (p[0] == 1).all() and all((t[0] == 0).all() for t in state.values())
    g[0][0] = 1.0
    g[0][1:256] = 1e-9
    ssd.adamw_step(p, g, state, step=2, lr=0.1, weight_decay=0.0)
    assert (state["exp_avg_sq"][0][1:256] == 1).all() and state["exp_avg_sq"][0][0] == 255
    assert (state["exp_avg_sq"][0][256:] == 0).all()


def test_past_32_bits(ssd):
    """A tensor of more than 2^32 elements: its last ones."""
    n = 2 ** 32 + 300
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    p, g = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))
    p[-600:] = torch.randn(600, device="cuda")
    g[-600:] = torch.randn(600, device="cuda")
    first = (n - 600) // 256 * 256
    a, b = p[first:].clone(), g[first:].clone()
    state, small = ssd.adamw_state(p, bits=8), ssd.adamw_state(a, bits=8)
    ssd.adamw_step(p, g, state, step=1, **HYPER)
    ssd.adamw_step(a, b, small, step=1, **HYPER)
    assert torch.equal(p[first:], a)
    assert torch.equal(state["exp_avg_scale"][0][first // 256:], small["exp_avg_scale"][0])
    v, w = state["exp_avg_sq"][0][first:].float(), small["exp_avg_sq"][0].float()
    assert (v - w).abs().max() <= 1      # the places differ, and so do the roundings
    del p, g, state
    torch.cuda.empty_cache()


def test_refusals(ssd):
    p, g, state = make([(10,), (20,)], F32, F32, 32, False)
    for kw in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0),
               dict(weight_decay=-0.1), dict(step=0), dict(lr=float("nan"))):
        with pytest.raises(RuntimeError, match="ARG"):
            ssd.adamw_step(p, g, state, **{**dict(step=1, lr=1e-3), **kw})
    norm = torch.ones((), device="cuda")
    for kw in (dict(max_norm=1.0), dict(grad_norm=norm), dict(grad_norm=norm.double(), max_norm=1.0),
               dict(step=norm), dict(lr=norm.double()), dict(lr=torch.ones(()))):
        with pytest.raises(ValueError):
            ssd.adamw_step(p, g, state, **{**dict(step=1, lr=1e-3), **kw})
    bad = [(p, g[:1], state), (p, [g[0], g[1][:5]], state), (p, [g[0], g[1].half()], state),
           (p, [g[0], g[1].cpu()], state), ([p[0], p[0]], [g[0], g[0]], state),
           (p, g, dict(state, exp_avg=state["exp_avg"][:1])),
           (p, g, dict(state, exp_avg=[t.double() for t in state["exp_avg"]])),
           (p, g, dict(state, master=[None, p[0]])), (p, g, ssd.adamw_state(p[:1])),
           (p, g, dict(ssd.adamw_state(p, bits=8), exp_avg_scale=None))]
    for a, b, s in bad:
        with pytest.raises(ValueError):
            ssd.adamw_step(a, b, s, step=1, lr=1e-3)
    same = [p[0], p[0]]
    with pytest.raises(ValueError, match="twice"):
        ssd.adamw_step(same, [g[0], g[0]], ssd.adamw_state(same), step=1, lr=1e-3)
    with pytest.raises(ValueError):
        ssd.adamw_state(p, bits=4)
    with pytest.raises(ValueError):
        ssd.adamw_moments(state, out=([t.clone() for t in p], [t.clone() for t in p]))
