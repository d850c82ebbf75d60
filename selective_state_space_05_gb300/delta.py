"""Python binding of the gated delta rule's C ABI (include/ssd_delta.h): the
chunked scan, its backward, a differentiable form of the two and the one-token
step.

Argument marshalling only, as in scan.py and block.py, whose conventions hold
here: ``delta_scan_fwd`` and ``delta_scan_bwd`` run on any stream and inside a
CUDA graph capture, ``delta_scan`` is a differentiable torch function of the
two, and tensors given to be written have their version counter moved on.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .block import _call, _chk, _empty, _float_dtype, _stream_of, _workspace
from .scan import _need, _ptr, _token_dense

_F32, _I32 = torch.float32, torch.int32


def delta_abi_version() -> int:
    return _lib.load().ssd_delta_abi_version()


def _strided(t: torch.Tensor, name: str, dtype, shape, dev) -> "_lib.Stride":
    """The strides of a [batch, seqlen, ...] tensor with dense tokens."""
    if not (t is not None and t.dtype is dtype and t.shape == shape and t.device == dev
            and _token_dense(t)):
        _need(t, name, dtype, shape, dev, strided=True)
    return _lib.Stride(t.stride(0), t.stride(1))


def _inputs(q, k, v, g, beta, scale, initial_states, seq_idx):
    """Checks what the scan and its backward take.  Returns the C call's
    arguments up to the sizes, the sizes, dtype code and device."""
    dt = _float_dtype(q, "q")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [batch, seqlen, ngroups, dstate] and v [batch, seqlen, "
                         "nheads, headdim]")
    dev, xd = q.device, q.dtype
    B, L, G, K = q.shape
    H, V = v.shape[2:]
    sq = _strided(q, "q", xd, q.shape, dev)
    sk = _strided(k, "k", xd, q.shape, dev)
    sv = _strided(v, "v", xd, (B, L, H, V), dev)
    _chk(g, "g", _F32, (B, L, H), dev)
    _chk(beta, "beta", _F32, (B, L, H), dev)
    if initial_states is not None:
        _chk(initial_states, "initial_states", _F32, (B, H, V, K), dev)
    if seq_idx is not None:
        _chk(seq_idx, "seq_idx", _I32, (B, L), dev)
    scale = K ** -0.5 if scale is None and K else float(scale or 0.0)
    args = (q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, g.data_ptr(), beta.data_ptr(),
            scale, _ptr(initial_states), _ptr(seq_idx))
    return args, (B, L, H, V, K, G), dt, dev


def _aligned(*tensors) -> int:
    """The C calls' `aligned` of [batch, seqlen, rows, columns] tensors."""
    for t in tensors:
        e, s, n = t.element_size(), t.stride(), t.shape
        if (t.data_ptr() | s[0] * e | s[1] * e | n[3] * e) & 15 or (
                n[0] > 1 and s[0] == 0) or (n[1] > 1 and s[1] == 0):
            return 0
    return 1


def delta_scan_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                   beta: torch.Tensor, *, scale: Optional[float] = None,
                   initial_states: Optional[torch.Tensor] = None,
                   seq_idx: Optional[torch.Tensor] = None, return_final_states: bool = False,
                   save: bool = False, out: Optional[torch.Tensor] = None,
                   final_states: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """The gated delta rule (ssd_delta_scan_fwd), per batch row and head:

        S' = exp(g_t) S_{t-1};  S_t = S' + beta_t (v_t - S' k_t) (outer) k_t
        out_t = scale * S_t q_t

    q, k [batch, seqlen, ngroups, dstate], v [batch, seqlen, nheads, headdim],
    fp32 or bf16, may be strided views whose tokens are dense; g (the decay's
    logarithm) and beta [batch, seqlen, nheads] fp32; states [batch, nheads,
    headdim, dstate] fp32; seq_idx [batch, seqlen] int32; scale defaults to
    dstate ** -0.5.  Returns out, or a tuple of out, with return_final_states
    the final states, and with save what delta_scan_bwd takes as `saved` (the
    workspace, which then must not be used for anything else).  final_states may
    be initial_states; otherwise outputs share no memory with inputs.  With bf16
    tensors the fp32 results (final states, dg, dbeta, d_initial_states) are off
    by 2e-6 to 6e-6 of their norm: factors are two bf16 terms."""
    args, sizes, dt, dev = _inputs(q, k, v, g, beta, scale, initial_states, seq_idx)
    B, L, H, V, K, G = sizes
    st = _stream_of(stream, dev)
    given = []
    if out is None:
        out = _empty((B, L, H, V), q.dtype, dev, stream)
    else:
        _chk(out, "out", q.dtype, (B, L, H, V), dev)
        given.append(out)
    if final_states is not None:
        _chk(final_states, "final_states", _F32, (B, H, V, K), dev)
        given.append(final_states)
    elif return_final_states:
        final_states = _empty((B, H, V, K), _F32, dev, stream)
    keep = 1 if save else 0
    ws, ws_bytes, hold = _workspace(
        _call("ssd_delta_scan_workspace_bytes")(B, L, H, V, K, G, dt, keep, _aligned(q, k, v)),
        workspace, dev, stream)
    code = _call("ssd_delta_scan_fwd")(*args, B, L, H, V, K, G, dt, out.data_ptr(),
                                       _ptr(final_states), keep, ws, ws_bytes, st)
    if code:
        _lib.check(code)
    if given:
        increment_version(given)
    res = (out,)
    if return_final_states:
        res += (final_states,)
    if save:
        res += (hold,)
    return res if len(res) > 1 else out


def delta_scan_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   g: torch.Tensor, beta: torch.Tensor, *, scale: Optional[float] = None,
                   initial_states: Optional[torch.Tensor] = None,
                   seq_idx: Optional[torch.Tensor] = None,
                   dfinal_states: Optional[torch.Tensor] = None,
                   saved: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of delta_scan_fwd (ssd_delta_scan_bwd) for the upstream
    gradients dout of out (dense) and dfinal_states of the final states (None:
    zero).  saved: what the forward on the same inputs returned with save, or
    None: it is computed again.  Returns dq, dk, dv in q's dtype, dg, dbeta
    fp32, and d_initial_states (None without initial_states)."""
    args, sizes, dt, dev = _inputs(q, k, v, g, beta, scale, initial_states, seq_idx)
    B, L, H, V, K, G = sizes
    xd = q.dtype
    _chk(dout, "dout", xd, (B, L, H, V), dev)
    if dfinal_states is not None:
        _chk(dfinal_states, "dfinal_states", _F32, (B, H, V, K), dev)
    if saved is not None:   # (of any type, as a workspace)
        _need(saved, "saved", device=dev)
    st = _stream_of(stream, dev)
    ws, ws_bytes, hold = _workspace(
        _call("ssd_delta_scan_bwd_workspace_bytes")(
            B, L, H, V, K, G, dt, int(saved is not None), _aligned(q, k, v, dout)),
        workspace, dev, stream)
    grads = dict(dq=_empty((B, L, G, K), xd, dev, stream), dk=_empty((B, L, G, K), xd, dev, stream),
                 dv=_empty((B, L, H, V), xd, dev, stream), dg=_empty((B, L, H), _F32, dev, stream),
                 dbeta=_empty((B, L, H), _F32, dev, stream),
                 d_initial_states=None if initial_states is None
                 else _empty((B, H, V, K), _F32, dev, stream))
    code = _call("ssd_delta_scan_bwd")(
        dout.data_ptr(), _ptr(dfinal_states), *args, B, L, H, V, K, G, dt, _ptr(saved),
        0 if saved is None else saved.numel() * saved.element_size(), *map(_ptr, grads.values()),
        ws, ws_bytes, st)
    if code:
        _lib.check(code)
    return grads


class _DeltaScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_states, seq_idx, scale, grad):
        ctx.set_materialize_grads(False)
        keep = grad and any(ctx.needs_input_grad)   # (set for leaves without grad mode too)
        ctx.empty = q.dim() == v.dim() == 4 and q.shape[0] * q.shape[1] == 0
        if ctx.empty:   # no token: answered without a launch (the explicit calls refuse it)
            _, (B, _, H, V, K, _), _, dev = _inputs(q, k, v, g, beta, scale, initial_states, seq_idx)
            _stream_of(None, dev)
            ctx.save_for_backward(q, k, v, g, beta, initial_states)
            return v.new_empty(v.shape), v.new_zeros((B, H, V, K), dtype=_F32) \
                if initial_states is None else initial_states.clone()
        out, final, *saved = delta_scan_fwd(q, k, v, g, beta, scale=scale,
                                            initial_states=initial_states, seq_idx=seq_idx,
                                            return_final_states=True, save=keep)
        if keep:
            ctx.save_for_backward(q, k, v, g, beta, initial_states, seq_idx, *saved)
        ctx.scale = scale
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dfinal):
        if ctx.empty:
            *ins, init = ctx.saved_tensors
            if init is not None and dfinal is None:
                dfinal = torch.zeros_like(init)
            return (*(t.new_empty(t.shape) for t in ins), None if init is None else dfinal, None,
                    None, None)
        q, k, v, g, beta, init, seq_idx, saved = ctx.saved_tensors
        dout = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if dout is None \
            else dout.contiguous()
        d = delta_scan_bwd(dout, q, k, v, g, beta, scale=ctx.scale, initial_states=init,
                           seq_idx=seq_idx, saved=saved,
                           dfinal_states=None if dfinal is None else dfinal.contiguous())
        return (*d.values(), None, None, None)


def delta_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
               beta: torch.Tensor, *, scale: Optional[float] = None,
               initial_states: Optional[torch.Tensor] = None,
               seq_idx: Optional[torch.Tensor] = None, return_final_states: bool = False):
    """delta_scan_fwd as a differentiable torch function: gradients for q, k,
    v, g, beta and initial_states, through out and the final states.  Returns
    out, or (out, final_states)."""
    out, final = _DeltaScan.apply(q, k, v, g, beta, initial_states, seq_idx, scale,
                                  torch.is_grad_enabled())
    return (out, final) if return_final_states else out


def delta_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                      beta: torch.Tensor, state: torch.Tensor, *, scale: Optional[float] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token per batch row of the gated delta rule (ssd_delta_decode_step):
    q, k [batch, ngroups, dstate], v [batch, nheads, headdim]; g, beta [batch,
    nheads] fp32; state [batch, nheads, headdim, dstate] fp32, moved on in
    place; out may be v.  Returns out [batch, nheads, headdim]."""
    dt = _float_dtype(q, "q")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q must be [batch, ngroups, dstate] and v [batch, nheads, headdim]")
    dev, xd, shape = q.device, q.dtype, v.shape
    B, G, K = q.shape
    _, H, V = shape
    _chk(q, "q", xd, q.shape, dev)
    _chk(k, "k", xd, q.shape, dev)
    _chk(v, "v", xd, (B, H, V), dev)
    _chk(g, "g", _F32, (B, H), dev)
    _chk(beta, "beta", _F32, (B, H), dev)
    _chk(state, "state", _F32, (B, H, V, K), dev)
    st = _stream_of(stream, dev)
    given = [state]
    if out is None:
        out = _empty(shape, xd, dev, stream)
    else:
        _chk(out, "out", xd, shape, dev)
        given.append(out)
    code = _call("ssd_delta_decode_step")(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        K ** -0.5 if scale is None and K else float(scale or 0.0), state.data_ptr(), B, H, V, K, G,
        dt, out.data_ptr(), st)
    if code:
        _lib.check(code)
    increment_version(given)
    return out
