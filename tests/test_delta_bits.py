"""The gated delta rule's accuracy for fp32 tensors: as good as three bf16 terms a
factor and sums rounded to nearest make it, and better than two terms would be."""
import pytest
import torch

import delta_testutil as du

F32 = torch.float32
SIZES = [(1, 32, 1, 1, 64, 64), (2, 33, 1, 3, 17, 65), (1, 129, 3, 3, 33, 64),
         (2, 200, 1, 4, 48, 48), (2, 100, 1, 2, 32, 32), (1, 70, 1, 2, 16, 24)]


def bound(K, V, products):
    """What a result may be off by, relative to its norm.  Each rounding is of an
    element by itself: one that truncates at 2^-23 is off by 2^-23 / sqrt(3) in the
    mean square, one to nearest by half of that; they are added as if all went the
    same way.  A product of a chain of `products`: its large terms' step is truncated
    twice (an mma's sixteen values in two halves), its steps' sums (of dstate / 16 or
    headdim / 16 steps, or of a chunk's two) are rounded to nearest.  The scores q k^T
    are summed in the tensor cores alone: dstate / 16 steps truncated.  Three decays'
    exponentials, two units of 2^-24 each, and three terms a factor, 2^-26 a factor."""
    nk, nv, truncated, nearest = -(-K // 16), -(-V // 16), 2.0 ** -23 / 3 ** 0.5, 2.0 ** -24 / 3 ** 0.5
    steps = 2 * nk + 7 + (0 if products <= 5 else nk + nv)
    return ((2 * products + nk) * truncated + steps * nearest + 3 * 2.0 ** -23
            + 2 * products * 2.0 ** -26)


FORWARD, BACKWARD = 5, 8      # S k, T y, the write, S q, P u; do P, dS k, dx T, ... on top
GRADS = ("dq", "dk", "dv", "d_initial_states")   # (dg and dbeta are sums of small parts)


def off(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


def case(B, L, G, H, V, K):
    d = du.inputs(B, L, G, H, V, K, F32, seed=L * 17 + V)
    gen = torch.Generator().manual_seed(3)
    dout, df = torch.randn(B, L, H, V, generator=gen), torch.randn(B, H, V, K, generator=gen)
    return d, dout, df, du.reference(d, dout, df)


def two_terms(x):
    x = x.double()
    hi = x.float().to(torch.bfloat16).double()
    return hi + (x - hi).float().to(torch.bfloat16).double()


@pytest.mark.parametrize("size", SIZES)
def test_two_terms_would_not_do(size):
    """The bound is below what is left when only the inputs, the state at each chunk's
    end and the result have two terms, and all else is computed in 64 bits."""
    (B, L, G, H, V, K) = size
    d, dout, df, (out, fin, grads) = case(*size)
    cut = {n: t if t is None or n in ("g", "beta", "seq_idx") else two_terms(t)
           for n, t in d.items()}
    outs, S = [], cut["initial_states"]
    for a in range(0, L, 32):
        part = {n: cut[n][:, a:a + 32].double() for n in du.NAMES}
        o, S = du.recurrence(dict(part, initial_states=two_terms(S), seq_idx=None))
        outs.append(two_terms(o))
    assert off(torch.cat(outs, 1), out) > 1.2 * bound(K, V, FORWARD)
    assert off(two_terms(S), fin) > 1.2 * bound(K, V, FORWARD)
    _, _, got = du.reference(cut, two_terms(dout), two_terms(df))
    for n in GRADS:
        assert off(two_terms(got[n]), grads[n]) > 1.2 * bound(K, V, BACKWARD), n


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
def test_three_terms_do(size):
    import selective_state_space_05_gb300 as ssd
    (B, L, G, H, V, K) = size
    d, dout, df, (out, fin, grads) = case(*size)
    c = du.to(d, "cuda")
    ins = tuple(c[n] for n in du.NAMES)
    o, f, saved = ssd.delta_scan_fwd(*ins, initial_states=c["initial_states"],
                                     return_final_states=True, save=True)
    assert off(o, out) <= bound(K, V, FORWARD)
    assert off(f, fin) <= bound(K, V, FORWARD)
    got = ssd.delta_scan_bwd(dout.cuda(), *ins, initial_states=c["initial_states"],
                             dfinal_states=df.cuda(), saved=saved)
    for n in GRADS:
        assert off(got[n], grads[n]) <= bound(K, V, BACKWARD), n
    # and of a gradient taken by differences, whose own error is far below
    gen = torch.Generator().manual_seed(4)
    base = {n: t if t is None else t.double() for n, t in d.items()}
    for n in ("q", "k", "v", "initial_states"):
        u = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        f = []
        for s in (1e-5, -1e-5):
            o, S = du.recurrence(dict(base, **{n: base[n] + s * u}))
            f.append((o * dout.double()).sum() + (S * df.double()).sum())
        g = got[("d_" if n == "initial_states" else "d") + n].double().cpu()
        diff = float(f[0] - f[1]) / 2e-5
        assert abs(float((g * u).sum()) - diff) <= bound(K, V, BACKWARD) * float(g.norm() * u.norm())
