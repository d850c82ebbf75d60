"""Definitions of the block's operators in 64 bits (torch on the CPU; their
gradients by autograd of these forwards) and the error bound the GPU tests
hold them to.

A bound has two parts: half a step of the output's type for its one rounding,
and `ops` fp32 roundings (2^-24 each) of `mag`, the sum of the magnitudes of
the terms that make the element up."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def assert_within(got, ref, mag, ops, what="", extra=0.0):
    """|got - ref| <= half a step of got's type * |ref| + ops * 2^-24 * mag +
    extra, element by element; NaN where ref is NaN."""
    half = half_step(got.dtype)
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaNs differ"
    e32 = (ops * U32 * mag + extra) * (1 + half)
    tiny = 2.0 ** -126   # below the normal range nothing is claimed
    bad = ((got - ref).abs() > half * ref.abs() + e32 + tiny) & ~torch.isnan(ref)
    if bad.any():
        i = int(torch.where(bad, ((got - ref).abs() / (half * ref.abs() + e32 + tiny)),
                            torch.zeros_like(ref)).argmax())
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst at {i}: got "
            f"{float(got.flatten()[i])}, want {float(ref.flatten()[i])}, bound "
            f"{float((half * ref.abs() + e32).flatten()[i])}")


def leaf(t):
    return None if t is None else t.detach().double().cpu().requires_grad_(True)


def silu(v):
    return v / (1 + torch.exp(-v))


def dsilu_mag(z):
    """Magnitude of the terms of silu'(z)."""
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z.abs() * (1 - s))


def add_rmsnorm(x, residual, weight, scale, eps):
    r = x if scale is None else x * scale
    if residual is not None:
        r = r + residual
    return weight * r / (r.square().mean(-1, keepdim=True) + eps).sqrt(), r


def gated_rmsnorm(y, z, weight, group_size, eps, before):
    gate = None if z is None else silu(z)
    u = y if before or z is None else y * gate
    n = u.unflatten(-1, (-1, group_size))
    n = (n / (n.square().mean(-1, keepdim=True) + eps).sqrt()).flatten(-2) * weight
    return n * gate if before and z is not None else n


def directional(f, args, i, d, h):
    """Central difference of sum-valued f along d in argument i."""
    lo, hi = list(args), list(args)
    lo[i], hi[i] = args[i] - h * d, args[i] + h * d
    return (f(*hi) - f(*lo)) / (2 * h)
