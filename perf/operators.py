"""Cases of the operators around the scan: the residual RMSNorm before a
block, the gated grouped RMSNorm after its scan, the causal conv1d's backward
and one-token step, the projections (matrix product with bias, activation and
residual) and the clipping of a gradient set by its global norm.

The large shapes are those of the 2.7B benchmark (80 heads of 64: 5120 inner
channels, one B/C group of state 128, so 5376 conv channels and 10576
projected ones, model width 2560, 8 x 4096 tokens); the fp32 projection is the
block of the worked example (width 2048, 4384 projected channels).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token for each of 8 sequences: the pre-norm of a decode step
        dict(name="add_rmsnorm step", op="add_rmsnorm", dtype="bf16", rows=8, dim=2560,
             scale=False, train=False),
        # the pre-norm of a training step, fp32 residual stream, learned residual scale
        dict(name="add_rmsnorm train", op="add_rmsnorm", dtype="bf16", rows=32768, dim=2560,
             scale=True, train=True),
        # the gated norm of a decode step: the gate is a slice of the projection
        dict(name="gated_rmsnorm step", op="gated_rmsnorm", dtype="bf16", rows=8, dim=5120,
             groups=1, before=False, train=False),
        # the gated norm of a training step, grouped, odd number of tokens
        dict(name="gated_rmsnorm train", op="gated_rmsnorm", dtype="bf16", rows=32765, dim=5120,
             groups=8, before=False, train=True),
        # conv of a decode step
        dict(name="conv1d step", op="conv1d_step", dtype="bf16", batch=8, channels=5376, width=4),
        # conv backward over packed documents, x a slice of the projection
        dict(name="conv1d backward", op="conv1d_bwd", dtype="bf16", batch=8, seqlen=4096,
             channels=5376, width=4, docs=5),
        # input projection of a decode step: bound by the weight's bytes
        dict(name="linear step", op="linear", dtype="bf16", rows=8, k=2560, n=10576, bias=False,
             act="none", residual="none", train=False),
        # output projection of a ragged prompt into the fp32 residual stream
        dict(name="linear prefill", op="linear", dtype="bf16", rows=1021, k=5120, n=2560,
             bias=True, act="none", residual="f32", train=False),
        # input projection of a training step, forward and both gradients
        dict(name="linear train", op="linear", dtype="bf16", rows=32768, k=2560, n=10576,
             bias=False, act="none", residual="none", train=True),
        # fp32 projection with bias and activation, forward and gradients
        dict(name="linear train f32", op="linear", dtype="f32", rows=4095, k=2048, n=4384,
             bias=True, act="silu", residual="none", train=True),
        # the ordinary step of a small model: the norm is below the limit, in place
        dict(name="clip small", op="clip", dtype="f32", blocks=2, width=512, place="in",
             clipped=False),
        # a large model whose bf16 gradients are clipped into the optimizer's fp32 ones
        dict(name="clip large", op="clip", dtype="bf16", blocks=16, width=2560, place="f32",
             clipped=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over its logarithm, a multiple of 8 three times in four."""
    v = _log(rng, lo, hi)
    return max(8, v // 8 * 8) if rng.random() < 0.75 else v


def draw(rng):
    op = rng.choice(["add_rmsnorm", "gated_rmsnorm", "conv1d_step", "conv1d_bwd", "linear",
                     "linear", "clip"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "add_rmsnorm":
        c.update(dim=_size(rng, 64, 8192), scale=rng.random() < 0.5, train=rng.random() < 0.6)
        c.update(rows=_log(rng, 1, min(32768, 32768 * 1280 // c["dim"])))
    elif op == "gated_rmsnorm":
        c.update(groups=rng.choice([1, 1, 2, 4, 8]), before=rng.random() < 0.4,
                 train=rng.random() < 0.6)
        c.update(dim=c["groups"] * _size(rng, 64, 8192 // c["groups"]))
        c.update(rows=_log(rng, 1, min(32768, 32768 * 2560 // c["dim"])))
    elif op == "conv1d_step":
        c.update(batch=_log(rng, 1, 256), channels=8 * _log(rng, 8, 1024), width=rng.randint(2, 5))
    elif op == "conv1d_bwd":
        c.update(batch=_log(rng, 1, 8), channels=8 * _log(rng, 8, 672), width=rng.randint(2, 5),
                 docs=rng.choice([1, 1, 3, 8]))
        c.update(seqlen=_log(rng, 1, 8192 // c["batch"]))
    elif op == "linear":
        c.update(rows=_log(rng, 1, 8192), k=_size(rng, 64, 6144), n=_size(rng, 64, 10576),
                 bias=rng.random() < 0.5, act=rng.choice(["none", "none", "silu", "gelu"]),
                 residual=rng.choice(["none", "none", "same", "f32"]), train=rng.random() < 0.5)
    else:
        c.update(blocks=_log(rng, 1, 12), width=_size(rng, 64, 2560),
                 place=rng.choice(["in", "same", "f32"]))
        c.update(clipped=c["place"] != "in")
    return c


def _clip_shapes(case):
    """The parameters of `blocks` Mamba-2 blocks of model width w: 2 w inner
    channels in heads of 64, a state of 128, conv of 4."""
    w = case["width"]
    inner, heads = 2 * w, max(1, 2 * w // 64)
    conv = inner + 256
    return [(2 * inner + 256 + heads, w), (w, inner), (conv, 4), (conv,), (heads,), (heads,),
            (heads,), (inner,), (w,)] * case["blocks"]


def _clip_sizes(case):
    return [math.prod(s) for s in _clip_shapes(case)]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def rnd(*shape, dt=torch.float32, by=1.0, plus=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by + plus).to(dt)

    s, op, t = dict(case=dict(case)), case["op"], DT[case["dtype"]]
    if op == "add_rmsnorm":
        r, d = case["rows"], case["dim"]
        s.update(x=rnd(r, d, dt=t), residual=rnd(r, d, by=3.0), weight=rnd(d, by=0.2, plus=1.0),
                 scale=rnd(d, by=0.1, plus=0.5) if case["scale"] else None)
        if case["train"]:
            s.update(dy=rnd(r, d, dt=t), dres=rnd(r, d))
    elif op == "gated_rmsnorm":
        r, d = case["rows"], case["dim"]
        proj = rnd(r, 2 * d + 336, dt=t)   # z | xBC | dt of the input projection
        s.update(y=rnd(r, d, dt=t, by=2.0), z=proj[:, :d], weight=rnd(d, by=0.2, plus=1.0))
        if case["train"]:
            s.update(dout=rnd(r, d, dt=t))
    elif op == "conv1d_step":
        b, c, w = case["batch"], case["channels"], case["width"]
        s.update(x=rnd(b, c, dt=t), conv_state=rnd(b, w - 1, c, dt=t),
                 weight=rnd(c, w, by=0.5), bias=rnd(c, by=0.2))
    elif op == "conv1d_bwd":
        b, l, c, w = case["batch"], case["seqlen"], case["channels"], case["width"]
        before = max(0, c - 256)           # the gate's channels stand before xBC
        proj = rnd(b, l, before + c + 80, dt=t)
        cut = torch.rand(b, case["docs"] - 1, generator=g, device="cuda") * l
        pos = torch.arange(l, device="cuda")
        seq = (pos[None, :, None] >= cut[:, None, :]).sum(-1).to(torch.int32)
        s.update(x=proj[:, :, before:before + c], weight=rnd(c, w, by=0.5), bias=rnd(c, by=0.2),
                 seq_idx=seq.contiguous() if case["docs"] > 1 else None,
                 dout=rnd(b, l, c, dt=t))
    elif op == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        rt = {"none": None, "same": t, "f32": torch.float32}[case["residual"]]
        s.update(x=rnd(m, k, dt=t), weight=rnd(n, k, dt=t, by=k ** -0.5),
                 bias=rnd(n, dt=t, by=0.2) if case["bias"] else None,
                 residual=rnd(m, n, dt=rt) if rt else None)
        if case["train"]:
            s.update(dout=rnd(m, n, dt=rt or t))
    else:
        sizes = _clip_sizes(case)
        flat = rnd(sum(sizes), dt=t, by=1e-3)
        ot = {"in": None, "same": t, "f32": torch.float32}[case["place"]]
        s.update(flat=flat, grads=list(flat.split(sizes)),
                 max_norm=(0.5 if case["clipped"] else 2.0) * 1e-3 * sum(sizes) ** 0.5)
        if ot is not None:
            into = torch.empty(sum(sizes), dtype=ot, device="cuda")
            s.update(into=into, out=list(into.split(sizes)))
    return s


# ------------------------------------------------------------ plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _act(name, v):
    if name == "silu":
        return v * _sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))
    return v


def _dact(name, v):
    if name == "silu":
        s = _sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(v * 0.5 ** 0.5))
                + v * torch.exp(-0.5 * v * v) * (2.0 * math.pi) ** -0.5)
    return torch.ones_like(v)


def _plain_add_rmsnorm(s):
    t, x, w = s["x"].dtype, s["x"].float(), s["weight"]
    r = s["residual"] + (x if s["scale"] is None else x * s["scale"])
    rstd = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    n = r * rstd
    o = dict(y=(n * w).to(t), residual_out=r)
    if "dy" in s:
        dy = s["dy"].float()
        a = dy * w
        dr = s["dres"] + rstd * (a - n * (a * n).mean(-1, keepdim=True))
        o.update(dresidual=dr, dweight=(dy * n).sum(0))
        if s["scale"] is None:
            o.update(dx=dr.to(t))
        else:
            o.update(dx=(dr * s["scale"]).to(t), dscale=(dr * x).sum(0))
    return o


def _plain_gated_rmsnorm(s):
    c, t, w = s["case"], s["y"].dtype, s["weight"]
    g = c["groups"]
    y, z = s["y"].float(), s["z"].float()
    sig = _sigmoid(z)
    gate = z * sig
    u = y if c["before"] else y * gate
    ug = u.unflatten(-1, (g, -1))
    rstd = 1.0 / torch.sqrt((ug * ug).mean(-1, keepdim=True) + EPS)
    n = (ug * rstd).flatten(-2)
    o = dict(out=(n * w * gate if c["before"] else n * w).to(t))
    if "dout" in s:
        do = s["dout"].float()
        dgate = sig * (1.0 + z * (1.0 - sig))
        dn = do * gate * w if c["before"] else do * w
        dng, ng = dn.unflatten(-1, (g, -1)), n.unflatten(-1, (g, -1))
        du = (rstd * (dng - ng * (dng * ng).mean(-1, keepdim=True))).flatten(-2)
        if c["before"]:
            o.update(dy=du.to(t), dz=(do * n * w * dgate).to(t), dweight=(do * n * gate).sum(0))
        else:
            o.update(dy=(du * gate).to(t), dz=(du * y * dgate).to(t), dweight=(do * n).sum(0))
    return o


def _plain_conv1d_step(s):
    t = s["x"].dtype
    win = torch.cat([s["conv_state"], s["x"][:, None]], 1)
    pre = (win.float() * s["weight"].t()).sum(1) + s["bias"]
    s["conv_state"].copy_(win[:, 1:])
    return dict(out=_act("silu", pre).to(t), conv_state=s["conv_state"])


def _ahead(v, w, fill=0.0):
    """[B, L, ...] -> [B, L, ..., w]: entry j is v at token t + j."""
    pad = torch.full_like(v[:, :1], fill).repeat_interleave(w - 1, 1)
    return torch.cat([v, pad], 1).unfold(1, w, 1)


def _behind(v, w, fill=0.0):
    """[B, L, ...] -> [B, L, ..., w]: entry k is v at token t - (w - 1) + k."""
    pad = torch.full_like(v[:, :1], fill).repeat_interleave(w - 1, 1)
    return torch.cat([pad, v], 1).unfold(1, w, 1)


def _plain_conv1d_bwd(s):
    t, w = s["x"].dtype, s["weight"]
    width = w.shape[1]
    taps = _behind(s["x"].float(), width)
    if s["seq_idx"] is not None:
        q = s["seq_idx"]
        taps = taps * (_behind(q, width, -1) == q[..., None])[:, :, None]
    pre = (taps * w).sum(-1) + s["bias"]
    dpre = s["dout"].float() * _dact("silu", pre)
    dw = (taps * dpre[..., None]).sum((0, 1))
    later = _ahead(dpre, width)
    if s["seq_idx"] is not None:
        later = later * (_ahead(q, width, -1) == q[..., None])[:, :, None]
    dx = (later * w.flip(1)).sum(-1)
    return dict(dx=dx.to(t), dweight=dw, dbias=dpre.sum((0, 1)))


def _plain_linear(s):
    c, t = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    pre = x @ w.t()
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    out = _act(c["act"], pre)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    o = dict(out=out.to(t if s["residual"] is None else s["residual"].dtype))
    if "dout" in s:
        dpre = s["dout"].float()
        if c["act"] != "none":
            dpre = dpre * _dact(c["act"], pre)
        o.update(dx=(dpre @ w).to(t), dweight=(dpre.t() @ x).to(t))
        if s["bias"] is not None:
            o.update(dbias=dpre.sum(0).to(t))
    return o


def _plain_clip(s):
    f = s["flat"].float()
    norm = torch.sqrt((f * f).sum())
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    into = s.get("into", s["flat"])
    into.copy_(f * coef)
    return dict(norm=norm, grads=into)


# ------------------------------------------------------------ the framework's calls

def _own(s):
    import selective_state_space_05_gb300 as ssd
    c = s["case"]
    op = c["op"]
    if op == "add_rmsnorm":
        y, r = ssd.add_rmsnorm_fwd(s["x"], s["residual"], s["weight"], scale=s["scale"], eps=EPS)
        o = dict(y=y, residual_out=r)
        if "dy" in s:
            b = ssd.add_rmsnorm_bwd(s["dy"], s["dres"], r, s["weight"], x=s["x"],
                                    scale=s["scale"], eps=EPS)
            o.update({k: v for k, v in b.items() if v is not None})
        return o
    if op == "gated_rmsnorm":
        kw = dict(group_size=c["dim"] // c["groups"], eps=EPS, norm_before_gate=c["before"])
        o = dict(out=ssd.gated_rmsnorm_fwd(s["y"], s["z"], s["weight"], **kw))
        if "dout" in s:
            o.update(ssd.gated_rmsnorm_bwd(s["dout"], s["y"], s["z"], s["weight"], **kw))
        return o
    if op == "conv1d_step":
        out = ssd.causal_conv1d_step(s["x"], s["conv_state"], s["weight"], s["bias"])
        return dict(out=out, conv_state=s["conv_state"])
    if op == "conv1d_bwd":
        return ssd.causal_conv1d_bwd(s["dout"], s["x"], s["weight"], s["bias"],
                                     seq_idx=s["seq_idx"])
    if op == "linear":
        act = None if c["act"] == "none" else c["act"]
        save = "dout" in s and act is not None
        out = ssd.linear_fwd(s["x"], s["weight"], s["bias"], activation=act,
                             residual=s["residual"], save_pre=save)
        out, pre = out if save else (out, None)
        o = dict(out=out)
        if "dout" in s:
            b = ssd.linear_bwd(s["dout"], s["x"], s["weight"], activation=act, pre=pre,
                               need_dbias=s["bias"] is not None)
            o.update({k: v for k, v in b.items() if v is not None})
        return o
    norm = ssd.clip_grads(s["grads"], s["max_norm"], out=s.get("out"))
    return dict(norm=norm, grads=s.get("into", s["flat"]))


PLAIN = {"add_rmsnorm": _plain_add_rmsnorm, "gated_rmsnorm": _plain_gated_rmsnorm,
         "conv1d_step": _plain_conv1d_step, "conv1d_bwd": _plain_conv1d_bwd,
         "linear": _plain_linear, "clip": _plain_clip}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "add_rmsnorm":
        n, d = case["rows"] * case["dim"], case["dim"]
        b = n * (2 * e + 8) + 4 * d * (2 if case["scale"] else 1)   # x, y, residual in and out
        f = 5 * n
        if case["train"]:   # dy, dresidual in; dresidual, dx out; the parameters' gradients
            b += n * (2 * e + 8) + 4 * d * (2 if case["scale"] else 1)
            f += 12 * n
        return dict(bytes=b, flops=f)
    if op == "gated_rmsnorm":
        n, d = case["rows"] * case["dim"], case["dim"]
        b, f = 3 * n * e + 4 * d, 10 * n
        if case["train"]:   # dout in; dy, dz out
            b, f = b + 3 * n * e + 4 * d, f + 25 * n
        return dict(bytes=b, flops=f)
    if op == "conv1d_step":
        n, w = case["batch"] * case["channels"], case["width"]
        return dict(bytes=n * e * 2 + 2 * n * (w - 1) * e + 4 * case["channels"] * (w + 1),
                    flops=n * (2 * w + 5))
    if op == "conv1d_bwd":
        n, w = case["batch"] * case["seqlen"] * case["channels"], case["width"]
        return dict(bytes=3 * n * e + 8 * case["channels"] * (w + 1)
                    + (4 * case["batch"] * case["seqlen"] if case["docs"] > 1 else 0),
                    flops=n * (6 * w + 10))
    if op == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        r = {"none": 0, "same": e, "f32": 4}[case["residual"]]
        b = (m * k + n * k) * e + m * n * ((r or e) + r) + (n * e if case["bias"] else 0)
        f = 2 * m * n * k
        if case["train"]:   # dout in; dx, dweight (and dbias) out
            b += m * n * (r or e) + (m * k + n * k) * e + (n * e if case["bias"] else 0)
            f += 4 * m * n * k
        return dict(bytes=b, flops=f)
    n = sum(_clip_sizes(case))
    o = {"in": 0, "same": e, "f32": 4}[case["place"]]
    return dict(bytes=n * (e + o) + 4, flops=3 * n)


# ------------------------------------------------------------ the definitions in 64 bits

def _exact_conv(x, w, b, seq):
    """Depthwise conv by its definition, from shifted copies of x."""
    width, out = w.shape[1], b.expand_as(x)
    for k in range(width):
        lag = width - 1 - k
        if lag >= x.shape[1]:
            continue
        tap = torch.nn.functional.pad(x[:, :x.shape[1] - lag], (0, 0, lag, 0))
        if seq is not None and lag:
            same = torch.zeros(seq.shape, dtype=x.dtype, device=x.device)
            same[:, lag:] = (seq[:, lag:] == seq[:, :-lag]).to(x.dtype)
            tap = tap * same[..., None]
        out = out + tap * w[:, k]
    return out


def exact(case, seed):
    """The definitions of the forwards in 64 bits, their gradients by
    automatic differentiation of those."""
    s, op, F = prepare(case, seed), case["op"], torch.nn.functional

    def leaf(v):
        return None if v is None else v.double().requires_grad_(True)

    if op == "add_rmsnorm":
        x, res, w, sc = leaf(s["x"]), leaf(s["residual"]), leaf(s["weight"]), leaf(s["scale"])
        r = res + (x if sc is None else sc * x)
        y = w * r / (r.square().mean(-1, keepdim=True) + EPS).sqrt()
        o = dict(y=y.detach(), residual_out=r.detach())
        if "dy" in s:
            names = dict(dx=x, dresidual=res, dweight=w, dscale=sc)
            names = {k: v for k, v in names.items() if v is not None}
            gr = torch.autograd.grad((y, r), list(names.values()),
                                     (s["dy"].double(), s["dres"].double()))
            o.update(zip(names, gr))
        return o
    if op == "gated_rmsnorm":
        y, z, w = leaf(s["y"]), leaf(s["z"]), leaf(s["weight"])
        u = y if case["before"] else y * F.silu(z)
        u = u.unflatten(-1, (case["groups"], -1))
        n = (u / (u.square().mean(-1, keepdim=True) + EPS).sqrt()).flatten(-2) * w
        out = n * F.silu(z) if case["before"] else n
        o = dict(out=out.detach())
        if "dout" in s:
            o.update(zip(("dy", "dz", "dweight"),
                         torch.autograd.grad(out, (y, z, w), s["dout"].double())))
        return o
    if op == "conv1d_step":
        full = torch.cat([s["conv_state"], s["x"][:, None]], 1)
        y = _exact_conv(full.double(), s["weight"].double(), s["bias"].double(), None)[:, -1]
        return dict(out=F.silu(y), conv_state=full[:, 1:].double())
    if op == "conv1d_bwd":
        x, w, b = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"])
        y = F.silu(_exact_conv(x, w, b, s["seq_idx"]))
        return dict(zip(("dx", "dweight", "dbias"),
                        torch.autograd.grad(y, (x, w, b), s["dout"].double())))
    if op == "linear":
        x, w, b = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"])
        out = F.linear(x, w, b)
        out = {"none": out, "silu": F.silu(out), "gelu": F.gelu(out)}[case["act"]]
        o = dict(out=out.detach() if s["residual"] is None
                 else out.detach() + s["residual"].double())
        if "dout" in s:
            names = dict(dx=x, dweight=w, dbias=b)
            names = {k: v for k, v in names.items() if v is not None}
            o.update(zip(names, torch.autograd.grad(out, list(names.values()),
                                                    s["dout"].double())))
        return o
    f = s["flat"].double()
    norm = f.square().sum().sqrt()
    return dict(norm=norm, grads=f * min(1.0, s["max_norm"] / (float(norm) + 1e-6)))
