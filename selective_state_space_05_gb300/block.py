"""Python binding of the block operators' C ABI (include/ssd_block.h): the
residual RMSNorm before a block and the gated grouped RMSNorm after its scan,
the projections with bias, activation and residual in their epilogue, with
their backwards and a differentiable form of each, the causal conv1d's backward
and one-token step, and gradient clipping.

Argument marshalling only, as in scan.py.  Each operator comes as
``<name>_fwd`` and ``<name>_bwd`` (explicit, usable on any stream and inside a
CUDA graph capture) and as ``<name>``, a differentiable torch function of the
two.  A backward that is captured into a CUDA graph should call ``<name>_bwd``:
capturing ``Tensor.backward`` ties the graph to autograd's own streams.

A tensor that is given to be written (out, residual_out, dx, dz, conv_state,
clipped gradients) has its version counter moved on, as torch's own in-place
functions do: a backward pass that saved its old value raises.  Replays of a
captured call are not counted.
"""
from __future__ import annotations

import array
import math
import operator
from typing import Optional

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .scan import _DT, _need, _ptr

_F32 = torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_fn = {}


def _call(name):
    """The library's function, looked up once."""
    f = _fn.get(name)
    if f is None:
        f = _fn[name] = getattr(_lib.load(), name)
    return f


def _chk(t, name, dtype, shape, dev) -> None:
    """A dense tensor of this dtype, shape and device (the checks of _need in
    one expression: a call of a few microseconds has several of them)."""
    if not (t is not None and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _need(t, name, dtype, shape, dev)


def _stream_of(stream, dev) -> int:
    """The cudaStream_t of `stream`, or of dev's current stream."""
    if dev.type != "cuda":
        raise ValueError("tensors must be CUDA tensors")
    if dev.index != _current_device():
        raise ValueError(f"tensors are on {dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return _raw_stream(dev.index)
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
        need = max(need, 256)
        given = _empty((need,), torch.uint8, dev, stream)
        return given.data_ptr(), need, given
    _need(given, "workspace", device=dev)
    return given.data_ptr(), given.numel() * given.element_size(), given


def _float_dtype(t: torch.Tensor, name: str) -> int:
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _no_rows(t: torch.Tensor) -> bool:
    """An empty batch: the differentiable forms answer it without a launch,
    with empty results and zero gradients of the parameters (the explicit calls
    refuse it, as the C ABI does)."""
    return t.numel() == 0 and t.dim() > 1 and t.shape[-1] > 0


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
    xd = x.dtype
    dt = _float_dtype(x, "x")
    dev, shape = x.device, x.shape
    dim = shape[-1] if shape else 0
    if residual is not None:
        residual_dtype = residual.dtype
        _chk(residual, "residual", residual_dtype, shape, dev)
    elif residual_dtype is None:
        residual_dtype = xd if residual_out is None else residual_out.dtype
    _chk(x, "x", xd, shape, dev)
    _chk(weight, "weight", _F32, (dim,), dev)
    if scale is not None:
        _chk(scale, "scale", _F32, (dim,), dev)
    st = _stream_of(stream, dev)
    given = []
    if out is None:
        out = _empty(shape, xd, dev, stream)
    else:
        _chk(out, "out", xd, shape, dev)
        given.append(out)
    if residual_out is None:
        residual_out = _empty(shape, residual_dtype, dev, stream)
    else:
        _chk(residual_out, "residual_out", residual_dtype, shape, dev)
        given.append(residual_out)
    code = _call("ssd_add_rmsnorm_fwd")(
        x.data_ptr(), _ptr(residual), _ptr(scale), weight.data_ptr(), eps,
        x.numel() // dim if dim else 0, dim, dt, _float_dtype(residual_out, "residual"),
        out.data_ptr(), residual_out.data_ptr(), st)
    if code:
        _lib.check(code)
    if given:
        increment_version(given)
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
    f32 = _F32
    _chk(dy, "dy", dy.dtype, shape, dev)
    rt = _float_dtype(residual_out, "residual_out")
    _chk(residual_out, "residual_out", residual_out.dtype, shape, dev)
    if dresidual_out is not None:
        _chk(dresidual_out, "dresidual_out", residual_out.dtype, shape, dev)
    _chk(weight, "weight", f32, (dim,), dev)
    if scale is not None:
        _chk(scale, "scale", f32, (dim,), dev)
        _chk(x, "x", dy.dtype, shape, dev)
    st = _stream_of(stream, dev)
    rows = dy.numel() // dim if dim else 0
    ws, ws_bytes, hold = _workspace(_call("ssd_add_rmsnorm_bwd_workspace_bytes")(rows, dim),
                                    workspace, dev, stream)
    dx = _empty(shape, dy.dtype, dev, stream) if need_dx else None
    dres = _empty(shape, residual_out.dtype, dev, stream) if need_dresidual else None
    dw = _empty((dim,), f32, dev, stream)
    ds = None if scale is None else _empty((dim,), f32, dev, stream)
    _lib.check(_call("ssd_add_rmsnorm_bwd")(
        _ptr(dy), _ptr(dresidual_out), _ptr(residual_out), None if scale is None else _ptr(x),
        _ptr(scale), _ptr(weight), float(eps), rows, dim, dt, rt, _ptr(dx), _ptr(dres), _ptr(dw),
        _ptr(ds), ws, ws_bytes, st))
    return dict(dx=dx, dresidual=dres, dweight=dw, dscale=ds)


class _AddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, scale, eps, residual_dtype):
        ctx.set_materialize_grads(False)
        if _no_rows(x):
            _float_dtype(x, "x")
            _stream_of(None, x.device)
            if residual is not None:
                residual_dtype = residual.dtype
                _chk(residual, "residual", residual_dtype, x.shape, x.device)
            _chk(weight, "weight", _F32, x.shape[-1:], x.device)
            if scale is not None:
                _chk(scale, "scale", _F32, x.shape[-1:], x.device)
            y, r = torch.empty_like(x), x.new_empty(x.shape, dtype=residual_dtype)
        else:
            y, r = add_rmsnorm_fwd(x, residual, weight, scale=scale, eps=eps,
                                   residual_dtype=residual_dtype)
        ctx.save_for_backward(r, weight, None if scale is None else x, scale)
        ctx.eps, ctx.has_residual, ctx.dtype = eps, residual is not None, x.dtype
        return y, r

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr):
        r, weight, x, scale = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(r.shape, dtype=ctx.dtype, device=r.device)
        if _no_rows(r):
            return (dy, torch.empty_like(r) if ctx.has_residual else None, torch.zeros_like(weight),
                    None if scale is None else torch.zeros_like(scale), None, None)
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

def _rows(t: torch.Tensor, name: str):
    """(batch, seqlen, strides) of a [..., channels] tensor with dense
    channels, whose rows are batch x seqlen at two strides."""
    shape, st = t.shape, t.stride()
    n = len(shape)
    if n == 0 or (shape[-1] > 1 and st[-1] != 1):
        raise ValueError(f"{name}: the channels of a token must be dense")
    if n == 3:
        return shape[0], shape[1], _lib.Stride(st[0], st[1])
    if n == 2:
        return 1, shape[0], _lib.Stride(0, st[0])
    if n == 1:
        return 1, 1, _lib.Stride(0, shape[0])
    # more: the outer dimensions have to be one evenly spaced dimension
    want = None
    for k, s in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if k == 1:
            continue
        if want is not None and s != want:
            raise ValueError(f"{name}: its rows must have one batch and one token stride")
        want = (s if want is None else want) * k
    batch = math.prod(shape[:-2])
    inner = next((s for k, s in zip(reversed(shape[:-2]), reversed(st[:-2])) if k > 1), 0)
    return batch, shape[-2], _lib.Stride(inner, st[-2])


def _chk_rows(t, name, dtype, shape, dev):
    """_rows of a tensor of this dtype, shape and device."""
    if not (t is not None and t.dtype is dtype and t.shape == shape and t.device == dev):
        if t is not None and t.is_cuda and t.device == dev and t.dtype is dtype:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        _need(t, name, dtype, shape, dev, strided=True)
    return _rows(t, name)


_NO_STRIDE = _lib.Stride(0, 0)


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
    yd, dev, shape = y.dtype, y.device, y.shape
    B, L, sy = _chk_rows(y, "y", yd, shape, dev)
    dim = shape[-1]
    sz, zp = _NO_STRIDE, None
    if z is not None:
        sz = _chk_rows(z, "z", yd, shape, dev)[2]
        zp = z.data_ptr()
    _chk(weight, "weight", _F32, (dim,), dev)
    st = _stream_of(stream, dev)
    given = out
    if out is None:
        out = _empty(shape, yd, dev, stream)
    else:
        _chk(out, "out", yd, shape, dev)
    code = _call("ssd_gated_rmsnorm_fwd")(
        y.data_ptr(), sy, zp, sz, weight.data_ptr(), eps, B, L, dim,
        dim if group_size is None else group_size, 1 if norm_before_gate else 0, dt,
        out.data_ptr(), st)
    if code:
        _lib.check(code)
    if given is not None:
        increment_version(given)
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
    yd, dev, shape = y.dtype, y.device, y.shape
    B, L, sy = _chk_rows(y, "y", yd, shape, dev)
    dim = shape[-1]
    _chk(dout, "dout", yd, shape, dev)
    _chk(weight, "weight", _F32, (dim,), dev)
    st = _stream_of(stream, dev)
    sz = sdz = _NO_STRIDE
    given = dz
    if z is not None:
        sz = _chk_rows(z, "z", yd, shape, dev)[2]
        if dz is None:
            dz = _empty(shape, yd, dev, stream)
        sdz = _chk_rows(dz, "dz", yd, shape, dev)[2]
    elif dz is not None:
        raise ValueError("dz is given without z")
    gs = dim if group_size is None else group_size
    ws, ws_bytes, hold = _workspace(_call("ssd_gated_rmsnorm_bwd_workspace_bytes")(B, L, dim, gs),
                                    workspace, dev, stream)
    dy = _empty(shape, yd, dev, stream)
    dw = _empty((dim,), _F32, dev, stream)
    _lib.check(_call("ssd_gated_rmsnorm_bwd")(
        dout.data_ptr(), y.data_ptr(), sy, _ptr(z), sz, weight.data_ptr(), eps, B, L, dim, gs,
        1 if norm_before_gate else 0, dt, dy.data_ptr(), _ptr(dz), sdz, dw.data_ptr(), ws,
        ws_bytes, st))
    if given is not None:
        increment_version(given)
    return dict(dy=dy, dz=dz, dweight=dw)


class _GatedRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, z, weight, group_size, eps, norm_before_gate):
        ctx.save_for_backward(y, z, weight)
        ctx.opts = dict(group_size=group_size, eps=eps, norm_before_gate=norm_before_gate)
        if _no_rows(y):
            _float_dtype(y, "y")
            _stream_of(None, y.device)
            if z is not None:
                _chk_rows(z, "z", y.dtype, y.shape, y.device)
            _chk(weight, "weight", _F32, y.shape[-1:], y.device)
            if group_size is not None and (group_size < 1 or y.shape[-1] % group_size):
                raise ValueError("group_size must divide the channels")
            return y.new_empty(y.shape)
        return gated_rmsnorm_fwd(y, z, weight, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, z, weight = ctx.saved_tensors
        if _no_rows(y):
            return (y.new_empty(y.shape), None if z is None else y.new_empty(y.shape),
                    torch.zeros_like(weight), None, None, None)
        g = gated_rmsnorm_bwd(dout.contiguous(), y, z, weight, **ctx.opts)
        return g["dy"], g["dz"], g["dweight"], None, None, None


def gated_rmsnorm(y: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor, *,
                  group_size: Optional[int] = None, eps: float = 1e-5,
                  norm_before_gate: bool = False) -> torch.Tensor:
    """gated_rmsnorm_fwd as a differentiable torch function: gradients for y,
    z and weight."""
    return _GatedRMSNorm.apply(y, z, weight, group_size, eps, norm_before_gate)


# --- causal conv1d: backward, one token --------------------------------------

def causal_conv1d_bwd(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                      bias: Optional[torch.Tensor] = None, *,
                      seq_idx: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
                      dx: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of causal_conv1d (ssd_causal_conv1d_bwd) for the upstream
    gradient dout; dout and x [batch, seqlen, channels] may be strided views
    with dense channels, and dx may be given as one (e.g. a slice of the
    projection's gradient).  Returns dx (x's dtype), dweight [channels, width]
    and dbias [channels] (fp32; None without bias)."""
    dt = _float_dtype(x, "x")
    if activation not in (None, "silu"):
        raise ValueError("activation must be None or 'silu'")
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, channels]")
    shape, xd, dev = x.shape, x.dtype, x.device
    Bsz, L, Cn = shape
    sx = _chk_rows(x, "x", xd, shape, dev)[2]
    sd = _chk_rows(dout, "dout", xd, shape, dev)[2]
    W = weight.shape[-1]
    _chk(weight, "weight", _F32, (Cn, W), dev)
    if bias is not None:
        _chk(bias, "bias", _F32, (Cn,), dev)
    if seq_idx is not None:
        _chk(seq_idx, "seq_idx", torch.int32, (Bsz, L), dev)
    st = _stream_of(stream, dev)
    given = dx
    if dx is None:
        dx = _empty(shape, xd, dev, stream)
    so = _chk_rows(dx, "dx", xd, shape, dev)[2]
    ws, ws_bytes, hold = _workspace(
        _call("ssd_causal_conv1d_bwd_workspace_bytes")(Bsz, L, Cn, W), workspace, dev, stream)
    dw = _empty((Cn, W), _F32, dev, stream)
    db = None if bias is None else _empty((Cn,), _F32, dev, stream)
    _lib.check(_call("ssd_causal_conv1d_bwd")(
        dout.data_ptr(), sd, x.data_ptr(), sx, weight.data_ptr(), _ptr(bias), _ptr(seq_idx), Bsz,
        L, Cn, W, int(activation == "silu"), dt, dx.data_ptr(), so, dw.data_ptr(), _ptr(db), ws,
        ws_bytes, st))
    if given is not None:
        increment_version(given)
    return dict(dx=dx, dweight=dw, dbias=db)


def causal_conv1d_step(x: torch.Tensor, conv_state: Optional[torch.Tensor], weight: torch.Tensor,
                       bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of causal_conv1d per batch row (ssd_causal_conv1d_step): x
    [batch, channels] (rows may be strided); conv_state [batch, width - 1,
    channels], the sequence's last inputs, oldest first, moved on in place
    (None for width 1).  Returns out [batch, channels]."""
    dt = _float_dtype(x, "x")
    if activation not in (None, "silu"):
        raise ValueError("activation must be None or 'silu'")
    if x.dim() != 2:
        raise ValueError("x must be [batch, channels]")
    shape, xd, dev = x.shape, x.dtype, x.device
    Bsz, Cn = shape
    if Cn > 1 and x.stride(1) != 1:
        raise ValueError("x: the channels of a token must be dense")
    W = weight.shape[-1]
    _chk(weight, "weight", _F32, (Cn, W), dev)
    if bias is not None:
        _chk(bias, "bias", _F32, (Cn,), dev)
    if W > 1:
        _chk(conv_state, "conv_state", xd, (Bsz, W - 1, Cn), dev)
    st = _stream_of(stream, dev)
    given = [conv_state] if W > 1 else []
    if out is None:
        out = _empty(shape, xd, dev, stream)
    else:
        _chk(out, "out", xd, shape, dev)
        given.append(out)
    code = _call("ssd_causal_conv1d_step")(
        x.data_ptr(), x.stride(0), conv_state.data_ptr() if W > 1 else None, weight.data_ptr(),
        _ptr(bias), Bsz, Cn, W, 1 if activation == "silu" else 0, dt, out.data_ptr(), st)
    if code:
        _lib.check(code)
    if given:
        increment_version(given)
    return out


class CausalConv1d(torch.autograd.Function):
    """causal_conv1d forward (scan.causal_conv1d), causal_conv1d_bwd backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, seq_idx, activation):
        from .scan import causal_conv1d
        ctx.save_for_backward(x, weight, bias, seq_idx)
        ctx.activation = activation
        return causal_conv1d(x, weight, bias, seq_idx=seq_idx, activation=activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x, weight, bias, seq_idx = ctx.saved_tensors
        g = causal_conv1d_bwd(dout.contiguous(), x, weight, bias, seq_idx=seq_idx,
                              activation=ctx.activation)
        return g["dx"], g["dweight"], g["dbias"], None, None


# --- projections --------------------------------------------------------------

_ACT = {None: 0, "silu": 1, "gelu": 2}
_PRE = {torch.bfloat16: torch.float16, torch.float32: torch.float32}


def _act_code(activation) -> int:
    code = _ACT.get(activation)
    if code is None:
        raise ValueError("activation must be None, 'silu' or 'gelu'")
    return code


def _row_stride(t: torch.Tensor, name: str) -> int:
    """The one stride between the rows of t seen as [rows, features]."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: each row must be dense")
    if t.is_contiguous() or t.dim() == 1:
        return t.shape[-1]
    step, want = None, None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = want = s
        if s != want:
            raise ValueError(f"{name}: its rows must be evenly spaced")
        want = s * n
    return t.shape[-1] if step is None else step


def _aligned(t: torch.Tensor, stride: int) -> bool:
    return t.data_ptr() % 16 == 0 and stride % 8 == 0


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
               save_pre: bool = False, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None):
    """out = act(x W^T + bias) + residual (ssd_linear_fwd).  x [..., in]
    (evenly spaced dense rows, e.g. a slice of a wider tensor), weight [out,
    in] and bias [out] of x's dtype; activation None, "silu" or "gelu";
    residual [..., out] fp32 or x's dtype, also evenly spaced; out may be the
    residual.  Returns out (the residual's dtype, x's without one), or (out,
    pre) with save_pre: the value before the activation for linear_bwd (fp16
    for bf16, fp32 for fp32)."""
    dt = _float_dtype(x, "x")
    act = _act_code(activation)
    dev, xd = x.device, x.dtype
    K = x.shape[-1]
    N = weight.shape[0]
    st = _stream_of(stream, dev)
    _chk(weight, "weight", xd, (N, K), dev)
    if bias is not None:
        _chk(bias, "bias", xd, (N,), dev)
    shape = x.shape[:-1] + (N,)
    sx = _row_stride(x, "x")
    sr, rt = 0, dt
    if residual is not None:
        if residual.shape != shape or residual.device != dev:
            raise ValueError(f"residual must have shape {tuple(shape)} on {dev}")
        rt = _float_dtype(residual, "residual")
        sr = _row_stride(residual, "residual")
    od = xd if residual is None else residual.dtype
    given = out
    if out is None:
        out = _empty(shape, od, dev, stream)
    else:
        _chk(out, "out", od, shape, dev)
    pre = _empty(shape, _PRE[xd], dev, stream) if save_pre else None
    rows = x.numel() // K if K else 0
    xp, wp = x.data_ptr(), weight.data_ptr()
    need = _call("ssd_linear_fwd_workspace_bytes")(
        rows, K, N, dt, 1 if (xp | wp) % 16 == 0 and sx % 8 == 0 else 0)
    ws, ws_bytes, hold = (None, 0, None) if need == 0 and workspace is None and rows > 0 else \
        _workspace(need, workspace, dev, stream)
    code = _call("ssd_linear_fwd")(
        xp, sx, wp, _ptr(bias), _ptr(residual), sr, rows, K, N, act, dt, rt, out.data_ptr(),
        _ptr(pre), ws, ws_bytes, st)
    if code:
        _lib.check(code)
    if given is not None:
        increment_version(given)
    return (out, pre) if save_pre else out


def linear_bwd(dout: torch.Tensor, x: Optional[torch.Tensor], weight: Optional[torch.Tensor], *,
               activation: Optional[str] = None, pre: Optional[torch.Tensor] = None,
               need_dx: bool = True, need_dweight: bool = True, need_dbias: bool = False,
               workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of linear_fwd (ssd_linear_bwd) for the dense upstream
    gradient dout, fp32 or x's dtype (dout is the residual's gradient as
    well).  pre is the forward's, with an activation.  Returns dx, dweight and
    dbias in x's dtype, None where not asked for."""
    given = x if x is not None else weight
    if given is None:
        raise ValueError("x or weight is required")
    dt = _float_dtype(given, "x")
    act = _act_code(activation)
    dev, xd = dout.device, given.dtype
    dd = _float_dtype(dout, "dout")
    st = _stream_of(stream, dev)
    _chk(dout, "dout", dout.dtype, dout.shape, dev)
    N, K = dout.shape[-1], given.shape[-1]
    rows = dout.numel() // N if N else 0
    shape = dout.shape[:-1] + (K,)
    if need_dx:
        _chk(weight, "weight", xd, (N, K), dev)
    sx = K
    if need_dweight:
        if x is None or x.shape != shape or x.device != dev:
            raise ValueError(f"x must have shape {tuple(shape)} on {dev}")
        sx = _row_stride(x, "x")
    if activation is not None:
        _chk(pre, "pre", _PRE[xd], dout.shape, dev)
    aligned = (dout.data_ptr() % 16 == 0 and (not need_dx or weight.data_ptr() % 16 == 0)
               and (not need_dweight or _aligned(x, sx)))
    ws, ws_bytes, hold = _workspace(
        _call("ssd_linear_bwd_workspace_bytes")(rows, K, N, dt, int(aligned),
                                                int(act == 0 and dd == dt)),
        workspace, dev, stream)
    dx = _empty(shape, xd, dev, stream) if need_dx else None
    dw = _empty((N, K), xd, dev, stream) if need_dweight else None
    db = _empty((N,), xd, dev, stream) if need_dbias else None
    _lib.check(_call("ssd_linear_bwd")(
        dout.data_ptr(), dd, x.data_ptr() if need_dweight else None, sx,
        weight.data_ptr() if need_dx else None, _ptr(pre) if act else None, rows, K, N, act, dt,
        _ptr(dx), _ptr(dw), _ptr(db), ws, ws_bytes, st))
    return dict(dx=dx, dweight=dw, dbias=db)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation):
        save = activation is not None and any(ctx.needs_input_grad[:3])
        ctx.empty = _no_rows(x)
        if ctx.empty:
            return _Linear.no_rows(ctx, x, weight, bias, residual, activation)
        got = linear_fwd(x, weight, bias, activation=activation, residual=residual, save_pre=save)
        out, pre = got if save else (got, None)
        ctx.save_for_backward(x if ctx.needs_input_grad[1] else None,
                              weight if ctx.needs_input_grad[0] else None, pre)
        ctx.activation, ctx.like = activation, (x.dtype, x.shape[-1])
        return out

    @staticmethod
    def no_rows(ctx, x, weight, bias, residual, activation):
        _float_dtype(x, "x")
        _act_code(activation)
        _stream_of(None, x.device)
        N = weight.shape[0]
        shape = x.shape[:-1] + (N,)
        _chk(weight, "weight", x.dtype, (N, x.shape[-1]), x.device)
        if bias is not None:
            _chk(bias, "bias", x.dtype, (N,), x.device)
        if residual is not None:
            _float_dtype(residual, "residual")
            if residual.shape != shape or residual.device != x.device:
                raise ValueError(f"residual must have shape {tuple(shape)} on {x.device}")
        ctx.save_for_backward(x, weight, bias)
        return x.new_empty(shape, dtype=x.dtype if residual is None else residual.dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        nx, nw, nb, nr = ctx.needs_input_grad[:4]
        if ctx.empty:
            x, weight, bias = ctx.saved_tensors
            return (x.new_empty(x.shape) if nx else None, torch.zeros_like(weight) if nw else None,
                    torch.zeros_like(bias) if nb else None, dout if nr else None, None)
        x, weight, pre = ctx.saved_tensors
        dout = dout.contiguous()
        g = dict(dx=None, dweight=None, dbias=None)
        if nx or nw or nb:
            # dbias alone needs neither operand: an empty one tells the type
            given = x if x is not None else weight
            if given is None:
                given = torch.empty((0, ctx.like[1]), dtype=ctx.like[0], device=dout.device)
            g = linear_bwd(dout, x if x is not None else given, weight,
                           activation=ctx.activation, pre=pre, need_dx=nx, need_dweight=nw,
                           need_dbias=nb)
        return g["dx"], g["dweight"], g["dbias"], dout if nr else None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           activation: Optional[str] = None,
           residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """linear_fwd as a differentiable torch function: gradients for x,
    weight, bias and residual."""
    return _Linear.apply(x, weight, bias, residual, activation)


# --- gradient norm and clipping ----------------------------------------------

def _storage_dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one block of memory (in any order of its
    dimensions), so that an element-wise pass may walk the block."""
    want = 1
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if s != want:
            return False
        want *= n
    return True


_dtype_of = operator.attrgetter("dtype")


def _tensor_table(tensors, name, dev):
    """Addresses of the tensors and their dtypes' codes (array.array), and
    whether all are contiguous.  (A model has hundreds of gradients: each check
    is one map over them.)"""
    ptrs = array.array("Q", map(torch.Tensor.data_ptr, tensors))
    try:
        codes = array.array("i", map(_DT.__getitem__, map(_dtype_of, tensors)))
    except KeyError as e:
        raise ValueError(f"{name}: tensors must be float32 or bfloat16, got {e.args[0]}") from None
    if set(map(torch.Tensor.get_device, tensors)) != {dev.index}:
        raise ValueError(f"{name}: the tensors must be on {dev}")
    contiguous = all(map(torch.Tensor.is_contiguous, tensors))
    if not contiguous:
        for t in tensors:
            if not (t.is_contiguous() or t.numel() == 0 or _storage_dense(t)):
                raise ValueError(f"{name}: tensors must be dense")
    return ptrs, codes, contiguous


def _address(a) -> int:
    """Where an array.array's items are (host memory; the array must live)."""
    return a.buffer_info()[0]


def _grad_list(grads):
    grads = [grads] if isinstance(grads, torch.Tensor) else [g for g in grads if g is not None]
    if not grads:
        raise ValueError("no gradients given")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("the gradients must be CUDA tensors")
    return grads, dev


def grad_norm(grads, *, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm over all elements of a tensor or an iterable of tensors
    (fp32 and bf16, None entries skipped; ssd_grad_norm), as a 0-d fp32
    tensor on their device."""
    grads, dev = _grad_list(grads)
    ptrs, codes, _ = _tensor_table(grads, "grads", dev)
    n = len(grads)
    sizes = array.array("q", map(torch.Tensor.numel, grads))
    st = _stream_of(stream, dev)
    ws, ws_bytes, hold = _workspace(_call("ssd_clip_grads_workspace_bytes")(n), workspace, dev,
                                    stream)
    norm = _empty((), _F32, dev, stream)
    _lib.check(_call("ssd_grad_norm")(
        _address(ptrs), _address(sizes), _address(codes), n, norm.data_ptr(), ws, ws_bytes, st))
    return norm


def clip_grads(grads, max_norm: float, *, eps: float = 1e-6, out=None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scales the gradients (a tensor or an iterable, None entries skipped) by
    min(1, max_norm / (norm + eps)) with their common 2-norm
    (ssd_clip_grads): in place, or into `out`, one tensor for each gradient
    that is not None, of its size and fp32 or bf16 (e.g. fp32 for an optimizer
    that takes bf16 gradients' clipped values so).  No host synchronisation.
    Returns the norm before clipping, 0-d fp32."""
    grads, dev = _grad_list(grads)
    ptrs, codes, dense = _tensor_table(grads, "grads", dev)
    n = len(grads)
    sizes = array.array("q", map(torch.Tensor.numel, grads))
    written, outs, out_codes = ptrs, None, None
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else [o for o in out if o is not None]
        if len(out) != n:
            raise ValueError(f"out has {len(out)} tensors for {n} gradients")
        outs, out_codes, dense_out = _tensor_table(out, "out", dev)
        written = outs
        if array.array("q", map(torch.Tensor.numel, out)) != sizes or (
                not (dense and dense_out)
                and any(o.shape != g.shape or o.stride() != g.stride()
                        for o, g in zip(out, grads))):
            raise ValueError("out must match its gradient's size (shape and strides, unless all "
                             "tensors are contiguous)")
    if len(set(written)) != n:
        full = [p for p, k in zip(written, sizes) if k]
        if len(set(full)) != len(full):
            raise ValueError("a tensor to write is given twice")
    st = _stream_of(stream, dev)
    ws, ws_bytes, hold = _workspace(_call("ssd_clip_grads_workspace_bytes")(n), workspace, dev,
                                    stream)
    norm = _empty((), _F32, dev, stream)
    _lib.check(_call("ssd_clip_grads")(
        _address(ptrs), _address(sizes), _address(codes), n,
        None if outs is None else _address(outs), None if outs is None else _address(out_codes),
        max_norm, eps, norm.data_ptr(), ws, ws_bytes, st))
    increment_version(grads if out is None else out)
    return norm
