"""The gated delta rule, the block's operators and the optimizer step together, as
examples/delta_block.py uses them: gradients of a whole block against the same
block in 64 bits, training steps against their definition, and decoding against one
call over the whole sequence."""
import copy
import importlib.util
import os

import pytest
import torch

import block_testutil as bt
import delta_testutil as dt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "delta_block.py")
    spec = importlib.util.spec_from_file_location("delta_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(block, p, hidden, residual, seq):
    """The block by its definitions; p: its parameters in 64 bits."""
    h, r = bt.add_rmsnorm(hidden, residual, p["norm"], None, 1e-5)
    z, qkv, a, b = block.split(h @ p["in_proj"].t())
    B, L, _ = qkv.shape
    out = torch.zeros_like(qkv) + p["conv_b"]
    for k in range(4):
        lag = 3 - k
        tap = qkv[:, :L - lag] * p["conv_w"][:, k]
        tap = torch.where((seq[:, lag:] == seq[:, :L - lag])[..., None], tap, torch.zeros_like(tap))
        out = out + torch.nn.functional.pad(tap, (0, 0, lag, 0))
    q, k, v = bt.silu(out).split([block.keys, block.keys, block.inner], dim=-1)
    unit = torch.full((block.keys,), block.dstate ** -0.5, dtype=torch.float64)
    q, k = (bt.gated_rmsnorm(t, None, unit, block.dstate, 1e-5, False).unflatten(
        -1, (block.groups, block.dstate)) for t in (q, k))
    g = -torch.exp(p["A_log"]) * torch.nn.functional.softplus(a + p["bias"])
    y, _ = dt.recurrence(dict(q=q, k=k, v=v.unflatten(-1, (block.heads, block.headdim)), g=g,
                              beta=torch.sigmoid(b), initial_states=None, seq_idx=seq))
    y = bt.gated_rmsnorm(y.flatten(-2), z, p["gnorm"], block.headdim, 1e-5, False)
    return y @ p["out_proj"].t(), r


def test_block_gradients(example):
    torch.manual_seed(1)
    block = example.Block(width=64, heads=4, headdim=24, groups=2, dstate=16)
    hidden = torch.randn(2, 77, 64, device="cuda", requires_grad=True)
    residual = torch.randn(2, 77, 64, device="cuda", requires_grad=True)
    seq = (torch.arange(77, device="cuda") // 30).int().repeat(2, 1).contiguous()
    out, r = block(hidden, residual, seq)
    do, dr = torch.randn_like(out), torch.randn_like(r)
    leaves = dict(block.named_parameters(), hidden=hidden, residual=residual)
    grads = torch.autograd.grad((out, r), list(leaves.values()), (do, dr))
    p = {k: bt.leaf(v) for k, v in leaves.items()}
    ref, _ = reference(block, p, p["hidden"], p["residual"], seq.cpu())
    want = torch.autograd.grad((ref, _), list(p.values()), (do.double().cpu(), dr.double().cpu()))
    # a step of the block is within 1e-5 (72 additions of 2^-23 in the scan, fewer
    # elsewhere); eight of them, forward and backward, and the norms' quotients
    assert (out.double().cpu() - ref).abs().max() <= 1e-4 * ref.abs().max()
    for k, a, b in zip(leaves, grads, want):
        assert (a.double().cpu() - b).abs().max() <= 2e-4 * b.abs().max(), k


def test_training_step(example):
    """A step of fp32 parameters against AdamW's definition in 64 bits, on gradients
    that are the same bits."""
    torch.manual_seed(2)
    model = example.Model(blocks=2)
    x = torch.randn(3, 50, 128, device="cuda")
    target = torch.roll(x, 1, dims=1)
    lr, eps, decay, most = 2e-3, 1e-8, 1e-2, 0.05
    other = copy.deepcopy(model)
    grads = torch.autograd.grad(example.loss_of(other, x, target), list(other.parameters()))
    norm = float(torch.cat([g.double().flatten() for g in grads]).norm())
    assert norm > most                      # clipping is at work
    _, got = example.train(model, x, target, steps=1, lr=lr, max_norm=most)
    assert abs(got[0] - norm) <= 1e-5 * norm
    for (k, p), q, g in zip(model.named_parameters(), other.parameters(), grads):
        g = g.double() * (most / (norm + 1e-6))
        # (the first step: both averages are the gradient's own)
        want = q.detach().double() * (1 - lr * decay) - lr * g / (g.abs() + eps)
        # the new value's rounding and the old one's product with 1 - lr decay; the
        # step, at most lr long, within 2^-18 of lr (root and quotient 2^-21, the averages
        # 2^-22, the norm 2^-20)
        bound = 2 * 2.0 ** -24 * q.detach().abs() + lr * 2.0 ** -18
        assert ((p.detach() - want).abs() <= bound).all(), k


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.bfloat16, 32),
                                        (torch.bfloat16, 8)])
def test_training_and_decoding(example, dtype, bits):
    torch.manual_seed(3)
    model = example.Model(blocks=2, dtype=dtype)
    x = torch.randn(3, 70, 128, device="cuda").to(dtype)
    before = copy.deepcopy(model)
    losses, norms = example.train(model, x, torch.roll(x.float(), 1, dims=1), steps=5, bits=bits)
    assert len(losses) == 5 and all(0 < n < float("inf") for n in losses + norms)
    for p, q in zip(model.parameters(), before.parameters()):
        assert torch.isfinite(p).all() and (p != q).any()
    with torch.no_grad():
        full = model(x)
    # fp32: as a block's outputs.  bf16: a block rounds six times on the way (the
    # projection, the conv, keys and queries, y twice, the output); a sum that differs in
    # its last bits may round to the next value, 2^-8 off
    tol = (1e-4 if dtype == torch.float32 else 12 * 2.0 ** -8) * full.abs().max()
    for prompt in (1, 2, 65):
        out, states = model.prefill(x[:, :prompt])
        assert (out - full[:, :prompt]).abs().max() <= tol
        for t in range(prompt, 70):
            assert (model.step(x[:, t], states) - full[:, t]).abs().max() <= tol
