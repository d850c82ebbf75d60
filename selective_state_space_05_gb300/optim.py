"""Python binding of the optimizer step's C ABI (include/ssd_optim.h): AdamW over
many tensors at once, its moments in fp32 or in 8 bits.

Argument marshalling only, as in block.py, next to whose ``grad_norm`` and
``clip_grads`` the step stands: given the gradients' norm it clips them as it
reads them.  Tensors that are written have their version counter moved on.
"""
from __future__ import annotations

import array
import ctypes
from typing import Optional

import torch
from torch.autograd.graph import increment_version

from . import _lib
from .block import _address, _call, _dtype_of, _empty, _storage_dense, _stream_of
from .scan import _DT

_F32, _I64 = torch.float32, torch.int64
BLOCK = 256   # values that share a scale of 8-bit moments

_ptr_of, _numel_of, _shape_of = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.size
_dev_of, _dense_of = torch.Tensor.get_device, torch.Tensor.is_contiguous


def optim_abi_version() -> int:
    return _lib.load().ssd_optim_abi_version()


def adamw_state(params, *, bits: int = 32, master: bool = False) -> dict:
    """Zero moments for adamw_step, for a list of parameters (fp32 or bf16): a
    dict of lists "exp_avg" and "exp_avg_sq" (bits 32: fp32 tensors like the
    parameters; bits 8: int8 and uint8 codes, with "exp_avg_scale" and
    "exp_avg_sq_scale", fp32, one for each 256 elements).  master: also fp32
    copies of the bf16 parameters, which the steps are then taken on."""
    params = [params] if isinstance(params, torch.Tensor) else list(params)
    if bits not in (32, 8):
        raise ValueError("bits must be 32 or 8")

    def like(dtype):
        return [torch.zeros_like(p, dtype=dtype, requires_grad=False) for p in params]

    state = dict(exp_avg=like(_F32 if bits == 32 else torch.int8),
                 exp_avg_sq=like(_F32 if bits == 32 else torch.uint8))
    if bits == 8:
        for n in ("exp_avg_scale", "exp_avg_sq_scale"):
            state[n] = [torch.zeros(-(-p.numel() // BLOCK), dtype=_F32, device=p.device)
                        for p in params]
    if master:
        state["master"] = [p.detach().to(_F32, copy=True) if p.dtype is torch.bfloat16 else None
                           for p in params]
    return state


def _table(tensors, name, dtypes, dev, sizes, of=_numel_of):
    """Addresses of the tensors, after checks of their sizes (None: any; of: what
    `sizes` lists, elements or shapes), device and type (dtypes: a type, or a dict
    of codes; then also the codes)."""
    if tensors is None:
        raise ValueError(f"{name} is required")
    if sizes is not None and list(map(of, tensors)) != sizes:
        raise ValueError(f"{name}: the tensors' number or sizes do not match the parameters'")
    if tensors and set(map(_dev_of, tensors)) != {dev.index}:
        raise ValueError(f"{name}: the tensors must be on {dev}")
    ptrs = array.array("Q", map(_ptr_of, tensors))
    if isinstance(dtypes, dict):
        kinds = set(map(_dtype_of, tensors))
        try:
            if len(kinds) == 1:
                return ptrs, array.array("i", [dtypes[kinds.pop()]]) * len(tensors)
            return ptrs, array.array("i", map(dtypes.__getitem__, map(_dtype_of, tensors)))
        except KeyError as e:
            raise ValueError(f"{name}: tensors must be float32 or bfloat16, got "
                             f"{e.args[0]}") from None
    if tensors and set(map(_dtype_of, tensors)) != {dtypes}:
        raise ValueError(f"{name}: the tensors must be {dtypes}")
    return ptrs, None


def _scales(tensors, name, dev, blocks):
    """Addresses of the 8-bit moments' scales: dense, one for each block."""
    ptrs, _ = _table(tensors, name, _F32, dev, blocks)
    if not all(map(_dense_of, tensors)):
        raise ValueError(f"{name}: tensors must be dense")
    return ptrs


def _same_layout(first, others) -> None:
    """The lists' tensors, of the same shapes, agree element by element: all
    contiguous, or dense with the first's strides."""
    if all(map(_dense_of, first)) and all(all(map(_dense_of, ts)) for _, ts in others):
        return
    for i, p in enumerate(first):
        if not (p.is_contiguous() or p.numel() == 0 or _storage_dense(p)):
            raise ValueError("the tensors must be dense")
        for name, ts in others:
            if not (ts[i].is_contiguous() and p.is_contiguous()) and \
                    ts[i].stride() != p.stride():
                raise ValueError(f"{name}: tensors must have their parameter's strides")


def _spread(values, places, n):
    """An array of n items, zero but for `values` at `places`."""
    full = array.array(values.typecode, bytes(n * values.itemsize))
    for i, x in zip(places, values):
        full[i] = x
    return full


def _empty_like(t, dev, stream):
    if t.is_contiguous():
        return _empty(t.shape, _F32, dev, stream)
    return torch.empty_like(t, dtype=_F32)


_STATE = ("exp_avg", "exp_avg_sq", "master", "exp_avg_scale", "exp_avg_sq_scale")


def _scalar(t, name, dtype, dev) -> int:
    if not (t.dtype is dtype and t.numel() == 1 and t.device == dev):
        raise ValueError(f"{name} must be one {dtype} value on {dev}")
    return t.data_ptr()


def _list(v):
    return v if isinstance(v, list) else [v] if isinstance(v, torch.Tensor) else list(v)


class _Options(ctypes.Structure):
    """ssd_adamw_t"""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_norm", ctypes.c_void_p),
                ("max_norm", ctypes.c_double), ("seed", ctypes.c_uint32)]


def adamw_step(params, grads, state: dict, *, step, lr, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 1e-2, grad_norm: Optional[torch.Tensor] = None,
               max_norm: Optional[float] = None, seed: int = 0, stream=None) -> None:
    """One AdamW step of all parameters, in place (ssd_adamw_step):

        m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
        p = p (1 - lr weight_decay)
            - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)

    params and grads: lists of fp32 or bf16 tensors of the same shapes (a gradient
    None leaves its parameter as it is); state: adamw_state's dict, whose moments
    (and masters) move on.  step: this step's number from 1, an int or one int64
    value on the device, which a captured graph reads again at each replay; lr: a
    number or one fp32 value on the device.  With grad_norm (what grad_norm() returned) and
    max_norm the gradients count as clip_grads would leave them in fp32, times
    min(1, max_norm / (grad_norm + 1e-6)), but are not written (an infinite norm
    makes that 0; clip_grads knows norms past fp32's range).  seed: of the 8-bit
    moments' rounding."""
    params, grads = _list(params), _list(grads)
    n = len(params)
    if len(grads) != n:
        raise ValueError(f"{len(grads)} gradients for {n} parameters")
    lists = {k: state.get(k) for k in _STATE}
    for k, ts in lists.items():
        if ts is not None and len(ts) != n:
            raise ValueError(f"{k} must have {n} tensors")
    have = None
    if any(g is None for g in grads):
        have = [i for i, g in enumerate(grads) if g is not None]
        params, grads = [params[i] for i in have], [grads[i] for i in have]
        lists = {k: ts if ts is None else [ts[i] for i in have] for k, ts in lists.items()}
    if not params:
        return
    dev = params[0].device
    if dev.type != "cuda":
        raise ValueError("the parameters must be CUDA tensors")
    st = _stream_of(stream, dev)
    m, v, master, ms, vs = lists.values()
    bits = 32 if ms is None and vs is None else 8
    sizes, shapes = array.array("q", map(_numel_of, params)), list(map(_shape_of, params))
    pp, pc = _table(params, "params", _DT, dev, None)
    gp, gc = _table(grads, "grads", _DT, dev, shapes, _shape_of)
    mp, _ = _table(m, "exp_avg", _F32 if bits == 32 else torch.int8, dev, shapes, _shape_of)
    vp, _ = _table(v, "exp_avg_sq", _F32 if bits == 32 else torch.uint8, dev, shapes, _shape_of)
    written = [*params, *m, *v]
    alike = [("grads", grads), ("exp_avg", m), ("exp_avg_sq", v)]
    tables, codes = [pp, gp, mp, vp], [pc, gc]
    if bits == 8:
        blocks = [-(-k // BLOCK) for k in sizes]
        for name, ts in (("exp_avg_scale", ms), ("exp_avg_sq_scale", vs)):
            tables.append(_scales(ts, name, dev, blocks))
            written += ts
    if master is not None:
        given = [i for i, w in enumerate(master) if w is not None]
        some = [master[i] for i in given]
        wp, _ = _table(some, "master", _F32, dev, [shapes[i] for i in given], _shape_of)
        alike.append(("master", some if len(given) == len(params) else
                      [params[i] if w is None else w for i, w in enumerate(master)]))
        tables.append(_spread(wp, given, len(params)))
        written += some
    _same_layout(params, alike)
    once = [pp, *tables[2:]]   # what is written
    if master is not None:
        once[-1] = wp
    if len(set().union(*once)) != sum(map(len, once)):
        full = [a for t in once for a in t if a]   # (0: no elements)
        if len(set(full)) != len(full):
            raise ValueError("a parameter or a tensor of the state is given twice")
    if have is not None:   # the others' places keep their numbers, with no elements
        tables = [_spread(t, have, n) for t in tables]
        codes = [_spread(t, have, n) for t in codes]
        sizes = _spread(sizes, have, n)
    at = [_address(t) for t in tables]
    opt = _Options(beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay,
                   seed=seed & 0xFFFFFFFF)
    if isinstance(step, torch.Tensor):
        opt.step_dev = _scalar(step, "step", _I64, dev)
    else:
        opt.step = step
    if isinstance(lr, torch.Tensor):
        opt.lr_dev = _scalar(lr, "lr", _F32, dev)
    else:
        opt.lr = lr
    if (grad_norm is None) != (max_norm is None):
        raise ValueError("grad_norm and max_norm go together")
    if grad_norm is not None:
        opt.grad_norm = _scalar(grad_norm, "grad_norm", _F32, dev)
        opt.max_norm = max_norm
    scales = at[4:6] if bits == 8 else (None, None)
    code = _call("ssd_adamw_step")(
        at[0], _address(codes[0]), at[1], _address(codes[1]), None if master is None else at[-1],
        at[2], at[3], *scales, _address(sizes), n, bits, ctypes.addressof(opt), st)
    if code:
        _lib.check(code)
    increment_version(written)


def adamw_moments(state: dict, *, out=None, stream=None):
    """The values that a state's moments stand for (ssd_adamw_moments for 8-bit
    ones): two lists of fp32 tensors, exp_avg's and exp_avg_sq's.  out: the two
    lists to write them to; without it moments in fp32 are returned themselves."""
    m, v = _list(state["exp_avg"]), _list(state["exp_avg_sq"])
    ms, vs = state.get("exp_avg_scale"), state.get("exp_avg_sq_scale")
    if ms is None and vs is None:
        if out is None:
            return m, v
        raise ValueError("out is for 8-bit moments: these are in fp32 already")
    if not m:
        return ([], []) if out is None else out
    dev = m[0].device
    if dev.type != "cuda":
        raise ValueError("the moments must be CUDA tensors")
    st = _stream_of(stream, dev)
    given = out is not None
    if not given:
        out = tuple([_empty_like(t, dev, stream) for t in ts] for ts in (m, v))
    om, ov = map(_list, out)
    sizes, shapes = array.array("q", map(_numel_of, m)), list(map(_shape_of, m))
    blocks = [-(-k // BLOCK) for k in sizes]
    tables = [_table(m, "exp_avg", torch.int8, dev, shapes, _shape_of)[0],
              _table(v, "exp_avg_sq", torch.uint8, dev, shapes, _shape_of)[0],
              _scales(ms, "exp_avg_scale", dev, blocks),
              _scales(vs, "exp_avg_sq_scale", dev, blocks),
              *(_table(ts, "out", _F32, dev, shapes, _shape_of)[0] for ts in (om, ov))]
    _same_layout(m, [("exp_avg_sq", v), ("out", om), ("out", ov)])
    code = _call("ssd_adamw_moments")(*map(_address, tables), _address(sizes), len(m), st)
    if code:
        _lib.check(code)
    if given:
        increment_version([*om, *ov])
    return om, ov
