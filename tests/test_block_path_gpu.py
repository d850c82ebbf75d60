"""The block's operators together, as examples/mamba2_block.py uses them:
gradients of a whole block against the same block in 64 bits, a training run,
and decoding against one call over the whole sequence."""
import importlib.util
import os

import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mamba2_block.py")
    spec = importlib.util.spec_from_file_location("mamba2_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(block, p, hidden, residual, seq):
    """The block by its definitions; p: its parameters in 64 bits."""
    h, r = bt.add_rmsnorm(hidden, residual, p["norm"], None, 1e-5)
    z, xbc, dt = block.split(h @ p["in_proj"].t())
    B, L, C = xbc.shape
    out = torch.zeros_like(xbc) + p["conv_b"]
    for k in range(4):
        lag = 3 - k
        tap = xbc[:, :L - lag] * p["conv_w"][:, k]
        tap = torch.where((seq[:, lag:] == seq[:, :L - lag])[..., None], tap, torch.zeros_like(tap))
        out = out + torch.nn.functional.pad(tap, (0, 0, lag, 0))
    x, Bm, Cm = block.heads_of(bt.silu(out))
    rep = block.heads // block.ngroups
    Bm, Cm = Bm.repeat_interleave(rep, 2), Cm.repeat_interleave(rep, 2)
    dt = torch.nn.functional.softplus(dt + p["dt_bias"])
    A = -torch.exp(p["A_log"])
    state = x.new_zeros(B, block.heads, block.headdim, block.dstate)
    ys = []
    for t in range(L):
        if t > 0:
            state = state * (seq[:, t] == seq[:, t - 1]).to(x.dtype)[:, None, None, None]
        state = state * torch.exp(dt[:, t] * A)[..., None, None] + (
            (dt[:, t, :, None] * x[:, t])[..., None] * Bm[:, t, :, None])
        ys.append((state * Cm[:, t, :, None]).sum(-1) + p["D"][:, None] * x[:, t])
    y = torch.stack(ys, 1).flatten(-2)
    g = bt.gated_rmsnorm(y, z, p["gnorm"], block.inner // block.ngroups, 1e-5, False)
    return g @ p["out_proj"].t(), r


def test_block_gradients(example):
    torch.manual_seed(1)
    block = example.Block(width=64, headdim=16, dstate=16, ngroups=2, chunk_size=16)
    hidden = torch.randn(2, 37, 64, device="cuda", requires_grad=True)
    residual = torch.randn(2, 37, 64, device="cuda", requires_grad=True)
    seq = (torch.arange(37, device="cuda") // 15).int().repeat(2, 1).contiguous()
    out, r = block(hidden, residual, seq)
    do, dr = torch.randn_like(out), torch.randn_like(r)
    leaves = dict(block.named_parameters(), hidden=hidden, residual=residual)
    grads = torch.autograd.grad((out, r), list(leaves.values()), (do, dr))
    p = {k: bt.leaf(v) for k, v in leaves.items()}
    ref, rr = reference(block, p, p["hidden"], p["residual"], seq.cpu())
    want = torch.autograd.grad((ref, rr), list(p.values()), (do.double().cpu(), dr.double().cpu()))
    # the scan's own tolerance for fp32 (1e-4 of the largest value) through a
    # block whose other steps are two orders below it
    assert (out.double().cpu() - ref).abs().max() <= 1e-4 * ref.abs().max()
    for k, a, b in zip(leaves, grads, want):
        assert (a.double().cpu() - b).abs().max() <= 2e-4 * b.abs().max(), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_and_decoding(example, dtype):
    torch.manual_seed(2)
    model = example.Model(blocks=2, dtype=dtype)
    x = torch.randn(3, 50, 128, device="cuda").to(dtype)
    losses, norms = example.train(model, x, torch.roll(x.float(), 1, dims=1), steps=12)
    assert losses[-1] < 0.9 * losses[0]
    assert all(n > 0 for n in norms)
    with torch.no_grad():
        full = model(x)
    tol = (1e-4 if dtype == torch.float32 else 2e-2) * full.abs().max()
    for prompt in (1, 2, 33):
        out, states = model.prefill(x[:, :prompt])
        assert (out - full[:, :prompt]).abs().max() <= tol
        for t in range(prompt, 50):
            assert (model.step(x[:, t], states) - full[:, t]).abs().max() <= tol
