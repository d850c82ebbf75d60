"""The gated delta rule by its definition, token by token in 64 bits on the CPU
(gradients by autograd of it), inputs for its tests, and their error bounds."""
from __future__ import annotations

import torch

NAMES = ("q", "k", "v", "g", "beta")


def inputs(B, L, G, H, V, K, dtype=torch.float32, seed=0, init=True, docs=None, strong=0.0):
    """Keys and queries of unit length, decays of a few percent to e^-2 a token
    (`strong`: the share of tokens with up to e^-30), beta in (0, 1).  docs:
    lengths of documents."""
    gen = torch.Generator().manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=gen)

    unit = torch.nn.functional.normalize
    d = dict(q=unit(rnd(B, L, G, K), dim=-1).to(dtype), k=unit(rnd(B, L, G, K), dim=-1).to(dtype),
             v=rnd(B, L, H, V).to(dtype), beta=torch.sigmoid(rnd(B, L, H)))
    u = torch.rand(B, L, H, generator=gen)
    d["g"] = -torch.exp(-4.0 + 4.7 * u)
    if strong:
        d["g"] -= 30.0 * torch.rand(B, L, H, generator=gen) * (
            torch.rand(B, L, H, generator=gen) < strong)
    d["initial_states"] = rnd(B, H, V, K) * 0.3 if init else None
    d["seq_idx"] = None
    if docs:
        assert sum(docs) == L
        d["seq_idx"] = torch.repeat_interleave(torch.arange(len(docs)), torch.tensor(docs)).to(
            torch.int32).expand(B, L).contiguous()
    return d


def to(d, device):
    return {k: None if v is None else v.to(device) for k, v in d.items()}


def recurrence(d, scale=None):
    """(out, final_states) in 64 bits of tensors in 64 bits."""
    q, k, v, g, beta = (d[n] for n in NAMES)
    B, L, H, V = v.shape
    r = H // q.shape[2]
    scale = q.shape[3] ** -0.5 if scale is None else scale
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    S = d["initial_states"]
    if S is None:
        S = v.new_zeros(B, H, V, q.shape[3])
    outs = []
    for t in range(L):
        decay = torch.exp(g[:, t])
        if d["seq_idx"] is not None and t > 0:
            decay = decay * (d["seq_idx"][:, t] == d["seq_idx"][:, t - 1])[:, None]
        S = S * decay[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None]
        outs.append((S * q[:, t, :, None]).sum(-1) * scale)
    return torch.stack(outs, 1), S


def leaves(d):
    """The inputs in 64 bits, those that have a gradient as leaves."""
    return {k: v if v is None or k == "seq_idx" else v.detach().double().cpu().requires_grad_(True)
            for k, v in d.items()}


def reference(d, dout=None, dfinal=None, scale=None):
    """out, final_states and the gradients' dict in 64 bits."""
    x = leaves(to(d, "cpu"))
    out, fin = recurrence(x, scale)
    if dout is None:
        return out.detach(), fin.detach()
    loss = (out * dout.double().cpu()).sum()
    if dfinal is not None:
        loss = loss + (fin * dfinal.double().cpu()).sum()
    names = [n for n in NAMES + ("initial_states",) if x[n] is not None]
    got = torch.autograd.grad(loss, [x[n] for n in names], allow_unused=True)
    grads = {("d_" if n == "initial_states" else "d") + n:
             torch.zeros_like(x[n]) if t is None else t for n, t in zip(names, got)}
    return out.detach(), fin.detach(), grads


# How far a result may be off, relative to its 2-norm.  A result is a chain of at
# most five products with ten factors.  bf16 inputs: a factor kept as two bf16
# terms is off by 2^-18, one product of terms that is left out by 2^-18: 20 of
# them.  fp32 inputs: three terms, 2^-26, and the products' fp32 sums, which the
# tensor cores truncate (2^-23 an addition): 128 / 16 + 32 / 16 + 32 / 16 steps of
# six products along the chain, 72 additions.
COMPUTE = {torch.bfloat16: 20 * 2.0 ** -18, torch.float32: 72 * 2.0 ** -23 + 20 * 2.0 ** -26}


def close(got, ref, dtype, what=""):
    """got (its own dtype) against ref in 64 bits, for inputs of `dtype`."""
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    norm = float(ref.norm())
    err = float((got - ref).norm())
    bound = (COMPUTE[dtype] + half) * norm + 1e-30
    assert err <= bound, f"{what}: off by {err / max(norm, 1e-300):.3g} of its norm, " \
                         f"bound {bound / max(norm, 1e-300):.3g}"
    # no single element far off: 32 times the whole's share of an element
    big = (got - ref).abs().max()
    rms = norm / max(1, ref.numel()) ** 0.5
    assert float(big) <= 32 * bound / max(1, ref.numel()) ** 0.5 + half * float(ref.abs().max()), \
        f"{what}: an element is off by {float(big):.3g}, rms {rms:.3g}"
