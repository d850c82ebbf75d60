"""Python binding of the block operators' C ABI (include/ssd_block.h): the
residual RMSNorm before a block and the gated grouped RMSNorm after its scan,
with their backwards and a differentiable form of each.

Argument marshalling only, as in scan.py.  Each operator comes as
``<name>_fwd`` and ``<name>_bwd`` (explicit, usable on any stream and inside a
CUDA graph capture) and as ``<name>``, a differentiable torch function of the
two.  A backward that is captured into a CUDA graph should call ``<name>_bwd``:
capturing ``Tensor.backward`` ties the graph to autograd's own streams.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .scan import _DT, _need, _ptr, _token_dense


def _stream_of(stream, dev) -> int:
    """The cudaStream_t of `stream`, or of dev's current stream."""
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, dev, stream) -> torch.Tensor:
    """Device memory for work on `stream`: allocated on that stream, so that
    the caching allocator does not hand it to another one while in use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(need: int, given: Optional[torch.Tensor], dev, stream):
    """(pointer, bytes, tensor that owns it) of a workspace of `need` bytes."""
    if given is None:
        given = _empty(max(need, 256), torch.uint8, dev, stream)
    else:
        _need(given, "workspace", device=dev)
    return given.data_ptr(), given.numel() * given.element_size(), given


def _float_dtype(t: torch.Tensor, name: str) -> int:
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def block_abi_version() -> int:
    return _lib.load().ssd_block_abi_version()


# --- residual RMSNorm --------------------------------------------------------

def add_rmsnorm_fwd(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, *,
                    scale: Optional[torch.Tensor] = None, eps: float = 1e-5,
                    residual_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None,
                    residual_out: Optional[torch.Tensor] = None, stream=None):
    """r = residual + scale * x, y = weight * r / rms(r)
    (ssd_add_rmsnorm_fwd).  x [..., dim]; residual the same shape, fp32 or x's
    dtype, or None (then r = scale * x, of residual_dtype, default x's);
    weight, scale [dim] fp32.  residual_out may be residual (in place).
    Returns (y, residual_out)."""
    dt = _float_dtype(x, "x")
    dev, shape = x.device, x.shape
    dim = shape[-1] if x.dim() else 0
    _need(x, "x", device=dev)
    if residual is not None:
        residual_dtype = residual.dtype
    elif residual_dtype is None:
        residual_dtype = x.dtype if residual_out is None else residual_out.dtype
    _need(residual, "residual", residual_dtype, shape, dev, optional=True)
    _need(weight, "weight", torch.float32, (dim,), dev)
    _need(scale, "scale", torch.float32, (dim,), dev, optional=True)
    st = _stream_of(stream, dev)
    if out is None:
        out = _empty(shape, x.dtype, dev, stream)
    else:
        _need(out, "out", x.dtype, shape, dev)
    if residual_out is None:
        residual_out = _empty(shape, residual_dtype, dev, stream)
    else:
        _need(residual_out, "residual_out", residual_dtype, shape, dev)
    _lib.check(_lib.load().ssd_add_rmsnorm_fwd(
        _ptr(x), _ptr(residual), _ptr(scale), _ptr(weight), float(eps),
        x.numel() // dim if dim else 0, dim, dt, _float_dtype(residual_out, "residual"),
        _ptr(out), _ptr(residual_out), st))
    return out, residual_out


def add_rmsnorm_bwd(dy: torch.Tensor, dresidual_out: Optional[torch.Tensor],
                    residual_out: torch.Tensor, weight: torch.Tensor, *,
                    x: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                    eps: float = 1e-5, need_dx: bool = True, need_dresidual: bool = True,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of add_rmsnorm_fwd (ssd_add_rmsnorm_bwd) for the upstream
    gradients dy of y and dresidual_out of residual_out (None: zero).  x is
    needed when scale is given.  Returns dx (dy's dtype), dresidual
    (residual_out's dtype), dweight and dscale (fp32), None where not asked
    for or without scale."""
    dt = _float_dtype(dy, "dy")
    dev, shape = dy.device, dy.shape
    dim = shape[-1] if dy.dim() else 0
    f32 = torch.float32
    _need(dy, "dy", device=dev)
    _need(residual_out, "residual_out", None, shape, dev)
    rt = _float_dtype(residual_out, "residual_out")
    _need(dresidual_out, "dresidual_out", residual_out.dtype, shape, dev, optional=True)
    _need(weight, "weight", f32, (dim,), dev)
    _need(scale, "scale", f32, (dim,), dev, optional=True)
    if scale is not None:
        _need(x, "x", dy.dtype, shape, dev)
    st = _stream_of(stream, dev)
    rows = dy.numel() // dim if dim else 0
    lib = _lib.load()
    ws, ws_bytes, hold = _workspace(int(lib.ssd_add_rmsnorm_bwd_workspace_bytes(rows, dim)),
                                    workspace, dev, stream)
    dx = _empty(shape, dy.dtype, dev, stream) if need_dx else None
    dres = _empty(shape, residual_out.dtype, dev, stream) if need_dresidual else None
    dw = _empty((dim,), f32, dev, stream)
    ds = None if scale is None else _empty((dim,), f32, dev, stream)
    _lib.check(lib.ssd_add_rmsnorm_bwd(
        _ptr(dy), _ptr(dresidual_out), _ptr(residual_out), None if scale is None else _ptr(x),
        _ptr(scale), _ptr(weight), float(eps), rows, dim, dt, rt, _ptr(dx), _ptr(dres), _ptr(dw),
        _ptr(ds), ws, ws_bytes, st))
    return dict(dx=dx, dresidual=dres, dweight=dw, dscale=ds)


class _AddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, scale, eps, residual_dtype):
        ctx.set_materialize_grads(False)
        y, r = add_rmsnorm_fwd(x, residual, weight, scale=scale, eps=eps,
                               residual_dtype=residual_dtype)
        ctx.save_for_backward(r, weight, None if scale is None else x, scale)
        ctx.eps, ctx.has_residual, ctx.dtype = eps, residual is not None, x.dtype
        return y, r

    @staticmethod
    def backward(ctx, dy, dr):
        r, weight, x, scale = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(r.shape, dtype=ctx.dtype, device=r.device)
        g = add_rmsnorm_bwd(dy.contiguous(), None if dr is None else dr.contiguous(), r, weight,
                            x=x, scale=scale, eps=ctx.eps, need_dx=ctx.needs_input_grad[0],
                            need_dresidual=ctx.has_residual and ctx.needs_input_grad[1])
        return g["dx"], g["dresidual"], g["dweight"], g["dscale"], None, None


def add_rmsnorm(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, *,
                scale: Optional[torch.Tensor] = None, eps: float = 1e-5,
                residual_dtype: Optional[torch.dtype] = None):
    """add_rmsnorm_fwd as a differentiable torch function: gradients for x,
    residual, weight and scale.  Returns (y, residual_out)."""
    return _AddRMSNorm.apply(x, residual, weight, scale, eps, residual_dtype)


# --- gated grouped RMSNorm ---------------------------------------------------

def _rows3(t: torch.Tensor) -> torch.Tensor:
    """[..., dim] as [batch, seqlen, dim] without a copy of dense channels."""
    if t.dim() == 3:
        return t
    if t.dim() == 2:
        return t.unsqueeze(0)
    if t.dim() == 1:
        return t.view(1, 1, -1) if t.is_contiguous() else t.reshape(1, 1, -1)
    return t.view(1, -1, t.shape[-1]) if t.is_contiguous() else t.flatten(0, -3)


def _stride3(t: Optional[torch.Tensor]) -> _lib.Stride:
    return _lib.Stride(0, 0) if t is None else _lib.Stride(t.stride(0), t.stride(1))


def _need_rows(t, name, dtype, shape, dev) -> None:
    """A [..., dim] tensor whose channels are dense; other strides are free."""
    _need(t, name, dtype, shape, dev, strided=True)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a token must be dense")


def gated_rmsnorm_fwd(y: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor, *,
                      group_size: Optional[int] = None, eps: float = 1e-5,
                      norm_before_gate: bool = False, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """RMSNorm over groups of group_size channels (default: all) with the gate
    silu(z), applied before the norm, or after it with norm_before_gate
    (ssd_gated_rmsnorm_fwd).  y, z [..., dim] (z None: no gate), channels
    dense, e.g. z a slice of the input projection; weight [dim] fp32.
    Returns a dense tensor of y's shape and dtype."""
    dt = _float_dtype(y, "y")
    dev, shape, dim = y.device, y.shape, y.shape[-1]
    _need_rows(y, "y", y.dtype, None, dev)
    if z is not None:
        _need_rows(z, "z", y.dtype, shape, dev)
    _need(weight, "weight", torch.float32, (dim,), dev)
    st = _stream_of(stream, dev)
    if out is None:
        out = _empty(shape, y.dtype, dev, stream)
    else:
        _need(out, "out", y.dtype, shape, dev)
    y3, z3 = _rows3(y), None if z is None else _rows3(z)
    _lib.check(_lib.load().ssd_gated_rmsnorm_fwd(
        _ptr(y3), _stride3(y3), _ptr(z3), _stride3(z3), _ptr(weight), float(eps), y3.shape[0],
        y3.shape[1], dim, dim if group_size is None else int(group_size),
        int(bool(norm_before_gate)), dt, _ptr(out), st))
    return out


def gated_rmsnorm_bwd(dout: torch.Tensor, y: torch.Tensor, z: Optional[torch.Tensor],
                      weight: torch.Tensor, *, group_size: Optional[int] = None,
                      eps: float = 1e-5, norm_before_gate: bool = False,
                      dz: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of gated_rmsnorm_fwd for the dense upstream gradient dout.
    dz may be given to have z's gradient written there (channels dense, e.g. a
    slice of the projection's gradient).  Returns dy (dense), dz (None without
    z) in y's dtype and dweight (fp32)."""
    dt = _float_dtype(y, "y")
    dev, shape, dim = y.device, y.shape, y.shape[-1]
    _need_rows(y, "y", y.dtype, None, dev)
    _need(dout, "dout", y.dtype, shape, dev)
    if z is not None:
        _need_rows(z, "z", y.dtype, shape, dev)
        if dz is None:
            dz = _empty(shape, y.dtype, dev, stream)
        _need_rows(dz, "dz", y.dtype, shape, dev)
    elif dz is not None:
        raise ValueError("dz is given without z")
    _need(weight, "weight", torch.float32, (dim,), dev)
    st = _stream_of(stream, dev)
    gs = dim if group_size is None else int(group_size)
    y3, z3, dz3 = _rows3(y), None if z is None else _rows3(z), None if z is None else _rows3(dz)
    if dz3 is not None and dz3.data_ptr() != dz.data_ptr():
        raise ValueError("dz: its rows must have one batch and one token stride")
    B, L = y3.shape[:2]
    lib = _lib.load()
    ws, ws_bytes, hold = _workspace(
        int(lib.ssd_gated_rmsnorm_bwd_workspace_bytes(B, L, dim, gs)), workspace, dev, stream)
    dy = _empty(shape, y.dtype, dev, stream)
    dw = _empty((dim,), torch.float32, dev, stream)
    _lib.check(lib.ssd_gated_rmsnorm_bwd(
        _ptr(dout), _ptr(y3), _stride3(y3), _ptr(z3), _stride3(z3), _ptr(weight), float(eps), B,
        L, dim, gs, int(bool(norm_before_gate)), dt, _ptr(dy), _ptr(dz3), _stride3(dz3), _ptr(dw),
        ws, ws_bytes, st))
    return dict(dy=dy, dz=dz, dweight=dw)


class _GatedRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, z, weight, group_size, eps, norm_before_gate):
        ctx.save_for_backward(y, z, weight)
        ctx.opts = dict(group_size=group_size, eps=eps, norm_before_gate=norm_before_gate)
        return gated_rmsnorm_fwd(y, z, weight, **ctx.opts)

    @staticmethod
    def backward(ctx, dout):
        y, z, weight = ctx.saved_tensors
        g = gated_rmsnorm_bwd(dout.contiguous(), y, z, weight, **ctx.opts)
        return g["dy"], g["dz"], g["dweight"], None, None, None


def gated_rmsnorm(y: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor, *,
                  group_size: Optional[int] = None, eps: float = 1e-5,
                  norm_before_gate: bool = False) -> torch.Tensor:
    """gated_rmsnorm_fwd as a differentiable torch function: gradients for y,
    z and weight."""
    return _GatedRMSNorm.apply(y, z, weight, group_size, eps, norm_before_gate)
