"""A Mamba-2 model of a few blocks, trained and then decoded token by token,
with every step of a block but A = -exp(A_log) in the library's kernels:

    h, residual = add_rmsnorm(hidden, residual)       the pre-norm and its stream
    z | xBC | dt = linear(h, in_proj)                 the input projection
    x | B | C = causal_conv1d(xBC)
    y = ssd_scan(x, dt, A, B, C)
    g = gated_rmsnorm(y, z)                           norm of y * silu(z)
    hidden = linear(g, out_proj)                      the output projection

Gradients flow through the same names (each is a differentiable function);
clip_grads bounds their norm before the optimizer's step.  A prompt leaves two
states per block, the conv's last inputs and the scan's, which
causal_conv1d_step and ssd_decode_step carry on one token at a time.

    python examples/mamba2_block.py          # needs a GPU and the built library
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_05_gb300 as ssd  # noqa: E402


class Block(torch.nn.Module):
    """One block of width `width`: heads of headdim channels, one group of
    dstate B/C channels, a conv of four taps."""

    def __init__(self, width=128, expand=2, headdim=32, dstate=64, ngroups=1, dtype=torch.float32,
                 device="cuda", chunk_size=64):
        super().__init__()
        self.inner, self.headdim, self.dstate, self.ngroups = expand * width, headdim, dstate, ngroups
        self.heads = self.inner // headdim
        self.conv_dim = self.inner + 2 * ngroups * dstate
        self.chunk = chunk_size
        f32 = dict(dtype=torch.float32, device=device)
        p = torch.nn.Parameter
        self.norm = p(torch.ones(width, **f32))
        self.in_proj = p((torch.randn(self.inner + self.conv_dim + self.heads, width, **f32)
                          * width ** -0.5).to(dtype))
        self.conv_w = p(torch.randn(self.conv_dim, 4, **f32) * 0.5)
        self.conv_b = p(torch.zeros(self.conv_dim, **f32))
        self.dt_bias = p(torch.full((self.heads,), -2.0, **f32))
        self.A_log = p(torch.log(torch.linspace(1, 8, self.heads, **f32)))
        self.D = p(torch.ones(self.heads, **f32))
        self.gnorm = p(torch.ones(self.inner, **f32))
        self.out_proj = p((torch.randn(width, self.inner, **f32) * self.inner ** -0.5).to(dtype))

    def split(self, proj):
        return proj.split([self.inner, self.conv_dim, self.heads], dim=-1)

    def heads_of(self, xbc):
        n = self.ngroups * self.dstate
        x, B, C = xbc.split([self.inner, n, n], dim=-1)
        return (x.unflatten(-1, (self.heads, self.headdim)),
                B.unflatten(-1, (self.ngroups, self.dstate)),
                C.unflatten(-1, (self.ngroups, self.dstate)))

    def forward(self, hidden, residual, seq_idx=None, last=False):
        """hidden [batch, seqlen, width], residual the fp32 stream (None before
        the first block).  Returns (hidden, residual); with `last`, the output
        projection closes the stream: (None, residual + hidden)."""
        h, residual = ssd.add_rmsnorm(hidden, residual, self.norm, residual_dtype=torch.float32)
        z, xbc, dt = self.split(ssd.linear(h, self.in_proj))
        x, B, C = self.heads_of(ssd.causal_conv1d(xbc, self.conv_w, self.conv_b, seq_idx=seq_idx))
        y = ssd.ssd_scan(x, dt, -torch.exp(self.A_log), B, C, chunk_size=self.chunk,
                         dt_bias=self.dt_bias, D=self.D, seq_idx=seq_idx)
        g = ssd.gated_rmsnorm(y.flatten(-2), z, self.gnorm, group_size=self.inner // self.ngroups)
        if last:
            return None, ssd.linear(g, self.out_proj, residual=residual)
        return ssd.linear(g, self.out_proj), residual

    @torch.no_grad()
    def prefill(self, hidden, residual, last=False):
        """forward over a prompt; also returns the states that step() carries on."""
        h, residual = ssd.add_rmsnorm_fwd(hidden, residual, self.norm,
                                          residual_dtype=torch.float32)
        z, xbc, dt = self.split(ssd.linear_fwd(h, self.in_proj))
        conv_state = xbc.new_zeros(xbc.shape[0], 3, self.conv_dim)
        kept = xbc[:, -3:]
        conv_state[:, 3 - kept.shape[1]:] = kept
        x, B, C = self.heads_of(ssd.causal_conv1d(xbc, self.conv_w, self.conv_b))
        y, state = ssd.ssd_scan_fwd(x, dt, -torch.exp(self.A_log), B, C, chunk_size=self.chunk,
                                    dt_bias=self.dt_bias, D=self.D, return_final_states=True)
        g = ssd.gated_rmsnorm_fwd(y.flatten(-2), z, self.gnorm,
                                  group_size=self.inner // self.ngroups)
        out = ssd.linear_fwd(g, self.out_proj, residual=residual if last else None)
        return (None, out) if last else (out, residual), (conv_state, state)

    @torch.no_grad()
    def step(self, hidden, residual, states, last=False):
        """One token per batch row, hidden [batch, width]; the states move on in
        place."""
        conv_state, state = states
        h, residual = ssd.add_rmsnorm_fwd(hidden, residual, self.norm,
                                          residual_dtype=torch.float32)
        z, xbc, dt = self.split(ssd.linear_fwd(h, self.in_proj))
        xbc = ssd.causal_conv1d_step(xbc, conv_state, self.conv_w, self.conv_b)
        x, B, C = self.heads_of(xbc)
        y = ssd.ssd_decode_step(x.contiguous(), dt.contiguous(), -torch.exp(self.A_log),
                                B.contiguous(), C.contiguous(), state, dt_bias=self.dt_bias,
                                D=self.D)
        g = ssd.gated_rmsnorm_fwd(y.flatten(-2), z, self.gnorm,
                                  group_size=self.inner // self.ngroups)
        out = ssd.linear_fwd(g, self.out_proj, residual=residual if last else None)
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


def train(model, inputs, targets, steps=20, lr=2e-3, max_norm=1.0, seq_idx=None):
    """A few AdamW steps on the mean squared error; returns losses and the
    gradients' norms before clipping."""
    params = list(model.parameters())
    opt = torch.optim.AdamW(params, lr=lr)
    losses, norms = [], []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = (model(inputs, seq_idx) - targets).square().mean()
        loss.backward()
        norms.append(ssd.clip_grads([p.grad for p in params], max_norm))
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


def main():
    torch.manual_seed(0)
    for dtype in (torch.float32, torch.bfloat16):
        model = Model(dtype=dtype)
        x = torch.randn(4, 96, 128, device="cuda").to(dtype)
        target = torch.roll(x.float(), 1, dims=1)     # the token before
        seq_idx = (torch.arange(96, device="cuda") // 40).int().repeat(4, 1).contiguous()
        losses, norms = train(model, x, target, seq_idx=seq_idx)
        print(f"{dtype}: loss {losses[0]:.4f} -> {losses[-1]:.4f}, "
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
