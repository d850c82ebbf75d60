"""A model of a few gated-delta-rule blocks, trained and then decoded token by
token, with every step of a block but its gates in the library's kernels:

    h, residual = add_rmsnorm(hidden, residual)       the pre-norm and its stream
    z | qkv | a | b = linear(h, in_proj)              the input projection
    q | k | v = causal_conv1d(qkv)
    q, k = gated_rmsnorm(.) / sqrt(dstate)            to unit length, a head each
    g = -exp(A_log) softplus(a + bias),  beta = sigmoid(b)
    y = delta_scan(q, k, v, g, beta)
    y = gated_rmsnorm(y, z)                           norm of y * silu(z), a head each
    hidden = linear(y, out_proj)                      the output projection

A training step ends with grad_norm and adamw_step, which clips the gradients as it
reads them.  A prompt leaves two states per block, the conv's last inputs and the
scan's, which causal_conv1d_step and delta_decode_step carry on one token at a time.

    python examples/delta_block.py          # needs a GPU and the built library
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_05_gb300 as ssd  # noqa: E402


class Block(torch.nn.Module):
    """One block of width `width`: heads of headdim values, groups of heads that
    share queries and keys of dstate channels, a conv of four taps."""

    def __init__(self, width=128, heads=4, headdim=64, groups=2, dstate=32, dtype=torch.float32,
                 device="cuda"):
        super().__init__()
        self.heads, self.headdim, self.groups, self.dstate = heads, headdim, groups, dstate
        self.inner, self.keys = heads * headdim, groups * dstate
        self.conv_dim = self.inner + 2 * self.keys
        f32 = dict(dtype=torch.float32, device=device)
        p = torch.nn.Parameter
        self.norm = p(torch.ones(width, **f32))
        self.in_proj = p((torch.randn(self.inner + self.conv_dim + 2 * heads, width, **f32)
                          * width ** -0.5).to(dtype))
        self.conv_w = p(torch.randn(self.conv_dim, 4, **f32) * 0.5)
        self.conv_b = p(torch.zeros(self.conv_dim, **f32))
        self.bias = p(torch.full((heads,), -2.0, **f32))
        self.A_log = p(torch.log(torch.linspace(1, 8, heads, **f32)))
        self.gnorm = p(torch.ones(self.inner, **f32))
        self.out_proj = p((torch.randn(width, self.inner, **f32) * self.inner ** -0.5).to(dtype))
        self.register_buffer("unit", torch.full((self.keys,), dstate ** -0.5, **f32))

    def split(self, proj):
        return proj.split([self.inner, self.conv_dim, self.heads, self.heads], dim=-1)

    def gates(self, a, b):
        """The decay's logarithm and the rate, fp32."""
        g = -torch.exp(self.A_log) * torch.nn.functional.softplus(a.float() + self.bias)
        return g, torch.sigmoid(b.float())

    def mixed(self, qkv, norm):
        """Queries, keys (of unit length) and values by heads."""
        q, k, v = qkv.split([self.keys, self.keys, self.inner], dim=-1)
        q, k = (norm(t, None, self.unit, group_size=self.dstate).unflatten(
            -1, (self.groups, self.dstate)) for t in (q, k))
        return q, k, v.unflatten(-1, (self.heads, self.headdim))

    def forward(self, hidden, residual, seq_idx=None, last=False):
        """hidden [batch, seqlen, width], residual the fp32 stream (None before
        the first block).  Returns (hidden, residual); with `last`, the output
        projection closes the stream: (None, residual + hidden)."""
        h, residual = ssd.add_rmsnorm(hidden, residual, self.norm, residual_dtype=torch.float32)
        z, qkv, a, b = self.split(ssd.linear(h, self.in_proj))
        qkv = ssd.causal_conv1d(qkv, self.conv_w, self.conv_b, seq_idx=seq_idx)
        q, k, v = self.mixed(qkv, ssd.gated_rmsnorm)
        y = ssd.delta_scan(q, k, v, *self.gates(a, b), seq_idx=seq_idx)
        y = ssd.gated_rmsnorm(y.flatten(-2), z, self.gnorm, group_size=self.headdim)
        if last:
            return None, ssd.linear(y, self.out_proj, residual=residual)
        return ssd.linear(y, self.out_proj), residual

    @torch.no_grad()
    def prefill(self, hidden, residual, last=False):
        """forward over a prompt; also returns the states that step() carries on."""
        h, residual = ssd.add_rmsnorm_fwd(hidden, residual, self.norm,
                                          residual_dtype=torch.float32)
        z, qkv, a, b = self.split(ssd.linear_fwd(h, self.in_proj))
        conv_state = qkv.new_zeros(qkv.shape[0], 3, self.conv_dim)
        kept = qkv[:, -3:]
        conv_state[:, 3 - kept.shape[1]:] = kept
        q, k, v = self.mixed(ssd.causal_conv1d(qkv, self.conv_w, self.conv_b),
                             ssd.gated_rmsnorm_fwd)
        y, state = ssd.delta_scan_fwd(q, k, v, *self.gates(a, b), return_final_states=True)
        y = ssd.gated_rmsnorm_fwd(y.flatten(-2), z, self.gnorm, group_size=self.headdim)
        out = ssd.linear_fwd(y, self.out_proj, residual=residual if last else None)
        return (None, out) if last else (out, residual), (conv_state, state)

    @torch.no_grad()
    def step(self, hidden, residual, states, last=False):
        """One token per batch row, hidden [batch, width]; the states move on in
        place."""
        conv_state, state = states
        h, residual = ssd.add_rmsnorm_fwd(hidden, residual, self.norm,
                                          residual_dtype=torch.float32)
        z, qkv, a, b = self.split(ssd.linear_fwd(h, self.in_proj))
        q, k, v = self.mixed(ssd.causal_conv1d_step(qkv, conv_state, self.conv_w, self.conv_b),
                             ssd.gated_rmsnorm_fwd)
        y = ssd.delta_decode_step(q, k, v.contiguous(), *self.gates(a, b), state)
        y = ssd.gated_rmsnorm_fwd(y.flatten(-2), z, self.gnorm, group_size=self.headdim)
        out = ssd.linear_fwd(y, self.out_proj, residual=residual if last else None)
        return (None, out) if last else (out, residual)


class Model(torch.nn.Module):
    def __init__(self, blocks=2, **kw):
        super().__init__()
        self.blocks = torch.nn.ModuleList(Block(**kw) for _ in range(blocks))

    def forward(self, hidden, seq_idx=None):
        residual = None
        for i, b in enumerate(self.blocks):
            hidden, residual = b(hidden, residual, seq_idx, last=i == len(self.blocks) - 1)
        return residual

    def prefill(self, hidden):
        hidden, residual, states = hidden.contiguous(), None, []
        for i, b in enumerate(self.blocks):
            (hidden, residual), s = b.prefill(hidden, residual, last=i == len(self.blocks) - 1)
            states.append(s)
        return residual, states

    def step(self, hidden, states):
        hidden, residual = hidden.contiguous(), None
        for i, b in enumerate(self.blocks):
            hidden, residual = b.step(hidden, residual, states[i], last=i == len(self.blocks) - 1)
        return residual


def loss_of(model, inputs, targets, seq_idx=None):
    return (model(inputs, seq_idx) - targets).square().mean()


def train(model, inputs, targets, steps=20, lr=2e-3, max_norm=1.0, bits=32, seq_idx=None):
    """A few AdamW steps, moments in `bits` bits, bf16 parameters with fp32 masters;
    returns losses and the gradients' norms before clipping."""
    params = list(model.parameters())
    state = ssd.adamw_state(params, bits=bits, master=True)
    losses, norms = [], []
    for i in range(steps):
        loss = loss_of(model, inputs, targets, seq_idx)
        grads = torch.autograd.grad(loss, params)
        norms.append(ssd.grad_norm(grads))
        ssd.adamw_step(params, grads, state, step=i + 1, lr=lr, grad_norm=norms[-1],
                       max_norm=max_norm, seed=i)
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


def main():
    torch.manual_seed(0)
    for dtype, bits in ((torch.float32, 32), (torch.bfloat16, 32), (torch.bfloat16, 8)):
        model = Model(dtype=dtype)
        x = torch.randn(4, 96, 128, device="cuda").to(dtype)
        target = torch.roll(x.float(), 1, dims=1)     # the token before
        seq_idx = (torch.arange(96, device="cuda") // 40).int().repeat(4, 1).contiguous()
        losses, norms = train(model, x, target, bits=bits, seq_idx=seq_idx)
        print(f"{dtype}, moments in {bits} bits: loss {losses[0]:.4f} -> {losses[-1]:.4f}, "
              f"gradient norm {norms[0]:.3f} -> {norms[-1]:.3f}")
        with torch.no_grad():
            full = model(x)
        out, states = model.prefill(x[:, :64])
        worst = (out - full[:, :64]).abs().max()
        for t in range(64, 96):
            worst = torch.maximum(worst, (model.step(x[:, t], states) - full[:, t]).abs().max())
        print(f"  64 tokens of prompt and 32 one by one against one call: max difference "
              f"{float(worst):.2e} of {float(full.abs().max()):.2f}")


if __name__ == "__main__":
    main()
