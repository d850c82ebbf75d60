"""The gated delta rule on the GPU against its recurrence in 64 bits."""
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


def check(ssd, d, dtype, dfinal=True, scale=None, seed=1):
    """Forward, gradients with and without what the forward keeps, one input."""
    ins, kw = split(d)
    B, L, H, V = d["v"].shape
    gen = torch.Generator().manual_seed(seed)
    dout = torch.randn(B, L, H, V, generator=gen).to(dtype)
    df = torch.randn(B, H, V, d["q"].shape[3], generator=gen) if dfinal else None
    want, fin, grads = du.reference(d, dout, df, scale)
    out, final, saved = ssd.delta_scan_fwd(*ins, scale=scale, return_final_states=True, save=True,
                                           **kw)
    du.close(out, want, dtype, "out")
    du.close(final, fin, dtype, "final_states")
    assert torch.equal(out, ssd.delta_scan_fwd(*ins, scale=scale, **kw))
    bkw = dict(scale=scale, dfinal_states=None if df is None else df.cuda(), **kw)
    got = ssd.delta_scan_bwd(dout.cuda(), *ins, saved=saved, **bkw)
    for n, ref in grads.items():
        du.close(got[n], ref, dtype, n)
    again = ssd.delta_scan_bwd(dout.cuda(), *ins, **bkw)
    for n in got:
        assert (got[n] is None and again[n] is None) or torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,G,H,V,K", [
    (1, 1, 1, 1, 16, 16), (2, 2, 1, 2, 1, 1), (1, 31, 2, 2, 8, 8), (1, 32, 1, 1, 64, 64),
    (2, 33, 1, 3, 17, 65), (1, 63, 2, 4, 130, 40), (1, 64, 1, 1, 128, 128), (3, 65, 2, 2, 24, 127),
    (1, 129, 3, 3, 33, 64), (2, 200, 1, 4, 48, 128), (1, 257, 2, 2, 200, 100)])
def test_sizes(ssd, dtype, B, L, G, H, V, K):
    check(ssd, du.inputs(B, L, G, H, V, K, dtype, seed=L * 131 + K), dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("docs", [[1] * 40, [31, 1, 1, 31, 1, 70], [64, 64, 7], [3, 130, 2]])
def test_documents(ssd, dtype, docs):
    check(ssd, du.inputs(2, sum(docs), 1, 2, 32, 32, dtype, seed=len(docs), docs=docs), dtype)
    check(ssd, du.inputs(1, sum(docs), 2, 2, 16, 64, dtype, init=False, docs=docs), dtype,
          dfinal=False, scale=0.7)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_decays(ssd, dtype):
    """Decays to e^-30 beside weak ones: those of the tokens after them keep
    their bits.  Below -104 the state starts anew, as in fp32."""
    check(ssd, du.inputs(1, 150, 2, 2, 32, 32, dtype, seed=5, strong=0.3), dtype)
    for low in (-105.0, -1e4, -float("inf")):
        d = du.inputs(1, 100, 1, 2, 32, 32, dtype, seed=6)
        e = du.inputs(1, 100, 1, 2, 32, 32, dtype, seed=6, docs=[7, 50, 43])
        d["g"][:, [7, 57]] = low
        e["g"][:, [7, 57]] = 0.0
        a, b = (ssd.delta_scan_fwd(*split(x)[0], return_final_states=True, **split(x)[1])
                for x in (d, e))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        dout = torch.ones_like(a[0])
        ga, gb = (ssd.delta_scan_bwd(dout, *split(x)[0], **split(x)[1]) for x in (d, e))
        for n in ga:
            assert torch.equal(ga[n], gb[n]), n
        assert (ga["dg"][:, [7, 57]] == 0).all()


def test_growing_and_plain_states(ssd):
    """g above 0 grows the state; beta 0 leaves it; g = 0 and beta = 1 is the
    rule without gates."""
    d = du.inputs(1, 90, 1, 2, 32, 48, F32, seed=8)
    d["g"] = d["g"].abs() * 0.05
    d["beta"][:, 20:40] = 0.0
    check(ssd, d, F32)
    d = du.inputs(1, 90, 1, 2, 32, 48, BF, seed=9)
    d["g"].zero_()
    d["beta"].fill_(1.0)
    check(ssd, d, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_views_of_a_projection(ssd, dtype, pad):
    """q, k and v as slices of one tensor, on and off 16 bytes."""
    B, L, G, H, V, K = 2, 70, 2, 4, 24, 40
    d = du.inputs(B, L, G, H, V, K, dtype, seed=11)
    parts = [d[n].flatten(2) for n in "qkv"]
    wide = torch.cat([torch.zeros(B, L, pad, dtype=dtype)] + parts, -1).cuda()
    q, k, v = wide[..., pad:].split([p.shape[-1] for p in parts], -1)
    q, k, v = q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V))
    assert not q.is_contiguous()
    ins, kw = split(d)
    dout = torch.randn(B, L, H, V, device="cuda").to(dtype)
    assert torch.equal(ssd.delta_scan_fwd(q, k, v, *ins[3:], **kw), ssd.delta_scan_fwd(*ins, **kw))
    a = ssd.delta_scan_bwd(dout, q, k, v, *ins[3:], **kw)
    b = ssd.delta_scan_bwd(dout, *ins, **kw)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    # a token for all rows, and a batch row for all
    one = d["k"][:, :1].cuda().expand(-1, L, -1, -1)
    assert torch.equal(ssd.delta_scan_fwd(ins[0], one, *ins[2:], **kw),
                       ssd.delta_scan_fwd(ins[0], one.contiguous(), *ins[2:], **kw))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pieces_of_a_sequence(ssd, dtype):
    """A sequence in pieces from final to initial states, then token by token,
    is the whole."""
    B, L, G, H, V, K = 2, 100, 2, 4, 40, 56
    d = du.inputs(B, L, G, H, V, K, dtype, seed=12)
    ins, kw = split(d)
    want, fin = du.reference(d)
    state, outs = kw["initial_states"], []
    for a, b in ((0, 1), (1, 30), (30, 80)):
        o, state = ssd.delta_scan_fwd(*(t[:, a:b].contiguous() for t in ins), initial_states=state,
                                      return_final_states=True)
        outs.append(o)
    state = state.clone()
    for t in range(80, L):
        outs.append(ssd.delta_decode_step(*(x[:, t].contiguous() for x in ins), state)[:, None])
    du.close(torch.cat(outs, 1), want, dtype, "out")
    du.close(state, fin, dtype, "state")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,G,H,V,K", [(1, 1, 1, 1, 1), (3, 2, 4, 33, 37), (2, 1, 2, 64, 128),
                                       (9, 3, 3, 100, 126), (1, 1, 1, 300, 4)])
def test_step(ssd, dtype, B, G, H, V, K):
    d = du.inputs(B, 1, G, H, V, K, dtype, seed=V + K)
    want, fin = du.reference(d)
    ins = [d[n][:, 0].contiguous().cuda() for n in du.NAMES]
    store = torch.empty(d["initial_states"].numel() + 1, device="cuda")
    for at in (0, 1):   # on and off 16 bytes
        state = store[at:at + d["initial_states"].numel()].view(d["initial_states"].shape)
        state.copy_(d["initial_states"])
        out = ssd.delta_decode_step(*ins, state)
        du.close(out, want[:, 0], dtype, "out")
        du.close(state, fin, F32, "state")
    assert state._version == 4     # the two copies into its store, and two steps


def test_step_keeps_infinities_to_their_rows(ssd):
    d = du.to(du.inputs(1, 1, 1, 2, 8, 16, F32, seed=3), "cuda")
    ins = [d[n][:, 0].contiguous() for n in du.NAMES]
    state, other = d["initial_states"].clone(), d["initial_states"].clone()
    ins[2][0, 0, 3] = float("nan")
    out = ssd.delta_decode_step(*ins, state)
    ins[2][0, 0, 3] = 0.0
    want = ssd.delta_decode_step(*ins, other)
    bad = torch.zeros(1, 2, 8, dtype=torch.bool, device="cuda")
    bad[0, 0, 3] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], want[~bad])
    assert torch.equal(torch.isnan(state).any(-1), bad) and torch.equal(state[~bad], other[~bad])


def test_gradient_against_differences(ssd):
    """The gradients in fp32 along random directions against central differences
    of the scan in 64 bits (truncation h^2, far below the bound)."""
    d = du.inputs(1, 70, 1, 2, 16, 24, F32, seed=21)
    ins, kw = split(d)
    dout = torch.randn(1, 70, 2, 16)
    got = ssd.delta_scan_bwd(dout.cuda(), *ins, **kw)
    base = {k: v if v is None else v.double() for k, v in d.items()}
    gen = torch.Generator().manual_seed(2)
    for n in du.NAMES + ("initial_states",):
        u = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        f = [(du.recurrence(dict(base, **{n: base[n] + s * h * u}))[0] * dout.double()).sum()
             for s in (1, -1)]
        diff = float(f[0] - f[1]) / (2 * h)
        g = got[("d_" if n == "initial_states" else "d") + n].double().cpu()
        assert abs(float((g * u).sum()) - diff) <= du.COMPUTE[F32] * float(g.norm() * u.norm()), n


def test_autograd(ssd):
    d = du.inputs(2, 50, 1, 2, 16, 24, F32, seed=30, docs=[20, 30])
    dout, df = torch.randn(2, 50, 2, 16), torch.randn(2, 2, 16, 24)
    _, _, want = du.reference(d, dout, df)
    c = du.to(d, "cuda")
    names = du.NAMES + ("initial_states",)
    ins = {n: c[n].requires_grad_(True) for n in names}
    out, fin = ssd.delta_scan(*(ins[n] for n in du.NAMES), initial_states=ins["initial_states"],
                              seq_idx=c["seq_idx"], return_final_states=True)
    loss = (out * dout.cuda()).sum() + (fin * df.cuda()).sum()
    for n, g in zip(names, torch.autograd.grad(loss, list(ins.values()), retain_graph=True)):
        du.close(g, want[("d_" if n == "initial_states" else "d") + n], F32, n)
    # only the final states, and only some inputs
    g = torch.autograd.grad((fin * df.cuda()).sum(), [ins["v"], ins["q"]])
    _, _, want = du.reference(d, torch.zeros_like(dout), df)
    du.close(g[0], want["dv"], F32, "dv")
    assert (g[1] == 0).all()
    with torch.no_grad():
        assert not ssd.delta_scan(*(ins[n] for n in du.NAMES)).requires_grad


def test_no_tokens(ssd):
    for B, L in ((0, 5), (2, 0)):
        d = du.inputs(B, L, 1, 2, 8, 16, BF)
        c = du.to(d, "cuda")
        ins = {n: c[n].requires_grad_(True) for n in du.NAMES + ("initial_states",)}
        out, fin = ssd.delta_scan(*(ins[n] for n in du.NAMES), return_final_states=True,
                                  initial_states=ins["initial_states"])
        assert out.shape == d["v"].shape and torch.equal(fin, c["initial_states"])
        (out.sum() + 2 * fin.sum()).backward()
        assert all(t.grad is not None and t.grad.shape == t.shape for t in ins.values())
        assert (ins["initial_states"].grad == 2).all()
        with pytest.raises(RuntimeError, match="ARG"):
            ssd.delta_scan_fwd(*(c[n] for n in du.NAMES))


def test_graph_streams_and_given_tensors(ssd):
    """A captured forward and backward, replayed on new inputs, two graphs whose
    workspaces are their own, a side stream, and outputs that are given."""
    d = [du.inputs(2, 130, 2, 2, 32, 64, BF, seed=s) for s in (40, 41)]
    (ins, kw), (ins2, kw2) = split(d[0]), split(d[1])
    dout = torch.randn(2, 130, 2, 32, device="cuda").to(BF)

    def run(i, k):
        o, f, saved = ssd.delta_scan_fwd(*i, return_final_states=True, save=True, **k)
        return [o, f] + list(ssd.delta_scan_bwd(dout, *i, saved=saved, **k).values())

    want, want2 = run(ins, kw), run(ins2, kw2)
    static, skw = [t.clone() for t in ins], {n: None if t is None else t.clone()
                                             for n, t in kw.items()}
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run(static, skw))
        graphs.append(graph)
    graphs[0].replay()
    graphs[1].replay()
    graphs[0].replay()
    for a, b, c in zip(want, got[0], got[1]):
        assert torch.equal(a, b) and torch.equal(a, c)
    for a, b in zip(static, ins2):
        a.copy_(b)
    skw["initial_states"].copy_(kw2["initial_states"])
    graphs[0].replay()
    for a, b in zip(want2, got[0]):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, fin = torch.empty_like(want[0]), torch.empty_like(want[1])
    o, f = ssd.delta_scan_fwd(*ins, out=out, final_states=fin, return_final_states=True,
                              stream=side, **kw)
    side.synchronize()
    assert o is out and f is fin and out._version == 1 and fin._version == 1
    assert torch.equal(out, want[0]) and torch.equal(fin, want[1])
    # an output off 16 bytes
    store = torch.zeros(out.numel() + 2, dtype=BF, device="cuda")
    view = store[1:-1].view(out.shape)
    ssd.delta_scan_fwd(*ins, out=view, **kw)
    assert torch.equal(view, out) and store[0] == 0 and store[-1] == 0


def test_long_sequences_keep_their_accuracy(ssd):
    """5000 tokens that hardly decay: the state's rounding does not add up."""
    for dtype in (BF, F32):
        d = du.inputs(1, 5000, 1, 1, 16, 32, dtype, seed=50)
        d["g"] *= 1e-3
        ins, kw = split(d)
        want, fin = du.reference(d)
        out, final = ssd.delta_scan_fwd(*ins, return_final_states=True, **kw)
        du.close(out, want, dtype, "out")
        du.close(final, fin, dtype, "final_states")


def test_refusals(ssd):
    d = du.to(du.inputs(1, 10, 1, 2, 16, 16, F32), "cuda")
    ins = [d[n] for n in du.NAMES]

    def swap(i, t):
        return [t if j == i else x for j, x in enumerate(ins)]

    for i, t in ((0, ins[0].half()), (1, ins[1].to(BF)), (2, ins[2].cpu()), (3, ins[3].double()),
                 (4, ins[4][:, :-1]), (1, ins[1][..., ::2]), (3, ins[3].transpose(1, 2))):
        with pytest.raises(ValueError):
            ssd.delta_scan_fwd(*swap(i, t))
    with pytest.raises(ValueError):
        ssd.delta_scan_fwd(*ins, initial_states=d["initial_states"].half())
    with pytest.raises(ValueError):
        ssd.delta_scan_fwd(*ins, seq_idx=torch.zeros(1, 10, dtype=torch.int64, device="cuda"))
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        ssd.delta_scan_fwd(*ins, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    out, saved = ssd.delta_scan_fwd(*ins, save=True)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        ssd.delta_scan_bwd(out, *ins, saved=saved[:-256])
    with pytest.raises(ValueError):
        ssd.delta_scan_bwd(out.transpose(1, 2), *ins)
    with pytest.raises(ValueError):
        ssd.delta_decode_step(*(x[:, 0] for x in ins), d["initial_states"].transpose(2, 3))


@pytest.mark.parametrize("V", [40, 130])
def test_more_sequences_than_sms(ssd, V):
    """So many heads that the SMs take their sequences in segments: every head is the
    same scan alone."""
    B, L, H, K = 4, 1500, 50, 32
    d = du.inputs(B, L, H, H, V, K, BF, seed=60)
    ins, kw = split(d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dout = torch.randn(B, L, H, V, generator=gen, device="cuda").to(BF)
    df = torch.randn(B, H, V, K, generator=gen, device="cuda")
    out, fin = ssd.delta_scan_fwd(*ins, return_final_states=True, **kw)
    got = ssd.delta_scan_bwd(dout, *ins, dfinal_states=df, **kw)
    for b, h in ((0, 0), (1, 17), (3, 49)):
        one = [t[b:b + 1, :, h:h + 1].contiguous() for t in ins]
        init = kw["initial_states"][b:b + 1, h:h + 1].contiguous()
        o, f = ssd.delta_scan_fwd(*one, initial_states=init, return_final_states=True)
        assert torch.equal(o[0, :, 0], out[b, :, h]) and torch.equal(f[0, 0], fin[b, h])
        g = ssd.delta_scan_bwd(dout[b:b + 1, :, h:h + 1].contiguous(), *one, initial_states=init,
                               dfinal_states=df[b:b + 1, h:h + 1].contiguous())
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(g[n][0, :, 0], got[n][b, :, h]), n
        assert torch.equal(g["d_initial_states"][0, 0], got["d_initial_states"][b, h])


@pytest.mark.parametrize("B,G,H,V,K,docs", [(1, 1, 1, 128, 128, None), (1, 2, 4, 40, 64, None),
                                            (2, 1, 1, 200, 100, [2000, 1, 2100]),
                                            (1, 3, 3, 130, 33, None)])
def test_a_few_long_sequences(ssd, B, G, H, V, K, docs):
    """Segments of a sequence all at once, joined by their effect on a state."""
    L = 4101
    d = du.inputs(B, L, G, H, V, K, BF, seed=70, docs=docs)
    d["g"] *= 0.02     # memory over many segments
    ins, kw = split(d)
    want, fin = du.reference(d)
    out, final, saved = ssd.delta_scan_fwd(*ins, return_final_states=True, save=True, **kw)
    du.close(out, want, BF, "out")
    du.close(final, fin, BF, "final_states")
    again = ssd.delta_scan_fwd(*ins, return_final_states=True, **kw)
    assert torch.equal(again[0], out) and torch.equal(again[1], final)
    # the backward takes what was kept, or runs it again
    dout = torch.ones_like(out)
    a = ssd.delta_scan_bwd(dout, *ins, saved=saved, **kw)
    b = ssd.delta_scan_bwd(dout, *ins, **kw)
    assert all(torch.equal(a[n], b[n]) for n in a)
    # and is that of the same sequence after its first tokens' pieces
    o1, s1 = ssd.delta_scan_fwd(*(t[:, :64].contiguous() for t in ins),
                                initial_states=kw["initial_states"], return_final_states=True)
    du.close(o1, want[:, :64], BF, "out of a short one")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_value_for_many(ssd, dtype):
    """Inputs expanded along the batch or the tokens (strides of 0)."""
    d = du.inputs(3, 70, 2, 4, 40, 48, dtype, seed=80)
    d["k"] = d["k"][:1].expand(3, -1, -1, -1)
    d["v"] = d["v"][:, :1].expand(-1, 70, -1, -1)
    ins, kw = split(d)
    ins = (ins[0], d["k"][:1].cuda().expand(3, -1, -1, -1),
           d["v"][:, :1].cuda().expand(-1, 70, -1, -1), *ins[3:])
    dout = torch.randn(3, 70, 4, 40, generator=torch.Generator().manual_seed(1)).to(dtype)
    want, fin, grads = du.reference(d, dout)
    out, saved = ssd.delta_scan_fwd(*ins, save=True, **kw)
    du.close(out, want, dtype, "out")
    got = ssd.delta_scan_bwd(dout.cuda(), *ins, saved=saved, **kw)
    for n, ref in grads.items():
        du.close(got[n], ref, dtype, n)
    # through autograd the leaf's gradient is the sum over what it was expanded along:
    # three (70) rounded gradients' sum, itself rounded
    leaf = [d["k"][:1].cuda().requires_grad_(), d["v"][:, :1].contiguous().cuda().requires_grad_()]
    o = ssd.delta_scan(ins[0], leaf[0].expand(3, -1, -1, -1), leaf[1].expand(-1, 70, -1, -1),
                       *ins[3:], **kw)
    o.backward(dout.cuda())
    for t, n, dim in ((leaf[0], "dk", 0), (leaf[1], "dv", 1)):
        ref = grads[n].sum(dim, keepdim=True)
        step = torch.finfo(dtype).eps / 2 * grads[n].abs().sum(dim, keepdim=True)
        off = (t.grad.double().cpu() - ref).abs()
        assert (off <= 72 * step + du.COMPUTE[dtype] * float(grads[n].norm())).all(), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [24, 130])
def test_values_that_are_not_finite_stay_in_their_head(ssd, dtype, V):
    """A head with a NaN and one with an infinity leave every other head's results as
    they are, whichever SM took them after the other."""
    B, L, H, K = 3, 200, 80, 40
    d = du.inputs(B, L, H, H, V, K, dtype, seed=81)
    ins, kw = split(d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dout = torch.randn(B, L, H, V, generator=gen, device="cuda").to(dtype)

    def both(ins):
        out, fin, saved = ssd.delta_scan_fwd(*ins, return_final_states=True, save=True, **kw)
        return dict(ssd.delta_scan_bwd(dout, *ins, saved=saved, **kw), out=out, fin=fin)

    clean = both(ins)
    bad = [t.clone() for t in ins]
    bad[2][0, 70, 7] = float("nan")
    bad[1][1, 130, 33] = float("inf")
    bad[3][2, 5, 60] = float("nan")
    got = both(bad)
    mask = torch.ones(B, H, dtype=torch.bool, device="cuda")
    for b, h in ((0, 7), (1, 33), (2, 60)):
        mask[b, h] = False
    for n, t in got.items():
        by_head = t if n in ("fin", "d_initial_states") else t.transpose(1, 2)
        ref = clean[n] if n in ("fin", "d_initial_states") else clean[n].transpose(1, 2)
        assert torch.equal(by_head[mask], ref[mask]), n
    assert not torch.isfinite(got["out"][0, 70:, 7]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_streams_at_once(ssd, dtype):
    """Two calls in flight beside each other, as often as it takes to meet."""
    jobs = []
    for seed, (B, L, H, V, K) in enumerate(((2, 900, 100, 64, 64), (1, 3000, 3, 40, 128))):
        ins, kw = split(du.inputs(B, L, H, H, V, K, dtype, seed=82 + seed))
        dout = torch.ones(B, L, H, V, device="cuda", dtype=dtype)
        jobs.append((ins, kw, dout))

    def run(ins, kw, dout):
        out, saved = ssd.delta_scan_fwd(*ins, save=True, **kw)
        return [out, *(t for t in ssd.delta_scan_bwd(dout, *ins, saved=saved, **kw).values())]

    want = [run(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for st, j in zip(streams, jobs):
            with torch.cuda.stream(st):
                got.append(run(*j))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_past_2_31_elements(ssd, dtype):
    """The last batch row of tensors of 2.35e9 elements is that row alone."""
    B, L, H, V, K = 7, 16384, 160, 128, 128
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB")
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*s):
        return torch.empty(s, dtype=dtype, device="cuda").normal_(generator=gen)

    q, k, v = rnd(B, L, H, K).mul_(K ** -0.5), rnd(B, L, H, K).mul_(K ** -0.5), rnd(B, L, H, V)
    g = -torch.rand(B, L, H, generator=gen, device="cuda")
    beta = torch.rand(B, L, H, generator=gen, device="cuda")
    ins = (q, k, v, g, beta)
    one = tuple(t[B - 1:].contiguous() for t in ins)
    o1, f1 = ssd.delta_scan_fwd(*one, return_final_states=True)
    out, fin = ssd.delta_scan_fwd(*ins, return_final_states=True)
    assert torch.isfinite(o1).all() and float(o1.abs().max()) > 0
    assert torch.equal(out[B - 1], o1[0]) and torch.equal(fin[B - 1], f1[0])
    if dtype is F32:
        return
    d1 = ssd.delta_scan_bwd(one[2], *one)
    got = ssd.delta_scan_bwd(v, *ins)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n][B - 1], d1[n][0]), n


@pytest.mark.parametrize("B,G,H,V,K,docs", [(1, 1, 2, 128, 128, None), (1, 2, 4, 40, 64, None),
                                            (2, 1, 1, 200, 100, [2000, 1, 1100])])
def test_gradients_of_a_few_long_sequences(ssd, B, G, H, V, K, docs):
    """The backward's segments all at once, with what was kept and without."""
    L = 3101
    d = du.inputs(B, L, G, H, V, K, BF, seed=90, docs=docs)
    d["g"] *= 0.02     # gradients from many segments away
    ins, kw = split(d)
    gen = torch.Generator().manual_seed(2)
    dout = torch.randn(B, L, H, V, generator=gen).to(BF)
    df = torch.randn(B, H, V, K, generator=gen)
    _, _, grads = du.reference(d, dout, df)
    _, saved = ssd.delta_scan_fwd(*ins, save=True, **kw)
    got = ssd.delta_scan_bwd(dout.cuda(), *ins, saved=saved, dfinal_states=df.cuda(), **kw)
    for n, ref in grads.items():
        du.close(got[n], ref, BF, n)
    again = ssd.delta_scan_bwd(dout.cuda(), *ins, dfinal_states=df.cuda(), **kw)
    assert all(torch.equal(got[n], again[n]) for n in got)
