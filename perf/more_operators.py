"""Cases of the gated delta rule (the chunked scan with its gradients and its
one-token step) and of the AdamW step over many tensors at once.

The large shapes have the inner width of the 2.7B benchmark (5120 channels, here
40 heads of 128 with a state of 128; 8 x 4096 tokens) and the parameters of its
blocks (model width 2560); others are generic.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64       # tokens a chunk of the plain form
BLOCK = 256      # values that share a scale of the 8-bit moments
BETAS, EPS, DECAY = (0.9, 0.999), 1e-8, 0.1


def listed():
    return [
        # one token for each of 8 sequences
        dict(name="delta step", op="step", dtype="bf16", batch=8, groups=40, heads=40, headdim=128,
             dstate=128),
        # one token for one sequence of a small model: latency
        dict(name="delta step one", op="step", dtype="f32", batch=1, groups=4, heads=8, headdim=64,
             dstate=64),
        # a ragged prompt that goes on from an earlier one's states, queries and keys shared by heads
        dict(name="delta prompt", op="fwd", dtype="bf16", batch=1, seqlen=1021, groups=20, heads=40,
             headdim=128, dstate=128, docs=1, init=True),
        # many sequences of packed documents, forward alone (evaluation)
        dict(name="delta forward", op="fwd", dtype="bf16", batch=8, seqlen=4096, groups=40, heads=40,
             headdim=128, dstate=128, docs=5, init=False),
        # one long sequence with few heads
        dict(name="delta long", op="fwd", dtype="bf16", batch=1, seqlen=32768, groups=16, heads=16,
             headdim=128, dstate=128, docs=1, init=False),
        # a training step's forward and backward
        dict(name="delta train", op="train", dtype="bf16", batch=4, seqlen=4096, groups=40, heads=40,
             headdim=128, dstate=128, docs=3, init=False),
        # the same in fp32: a small model, odd sizes, initial states that want a gradient
        dict(name="delta train f32", op="train", dtype="f32", batch=3, seqlen=777, groups=4, heads=8,
             headdim=64, dstate=72, docs=1, init=True),
        # the parameters of a small model in fp32
        dict(name="adamw small", op="adamw", param="f32", grad="f32", bits=32, blocks=2, width=512,
             clip=False),
        # a large one: bf16 parameters with fp32 masters, bf16 gradients clipped by their norm
        dict(name="adamw large", op="adamw", param="bf16", grad="bf16", bits=32, blocks=16,
             width=2560, clip=True),
        # moments in 8 bits
        dict(name="adamw 8 bits", op="adamw", param="bf16", grad="f32", bits=8, blocks=4, width=2560,
             clip=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "train", "train", "adamw"])
    if op == "adamw":
        c = dict(op=op, param=rng.choice(["bf16", "f32"]), grad=rng.choice(["bf16", "f32"]),
                 bits=rng.choice([32, 8]), width=8 * _log(rng, 8, 320), clip=rng.random() < 0.5)
        c.update(blocks=_log(rng, 1, 6))
        return c
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]),
             headdim=rng.choice([16, 32, 64, 64, 96, 128, 128, rng.randint(1, 160)]),
             dstate=rng.choice([16, 32, 64, 64, 128, 128, 128, rng.randint(1, 128)]))
    c["groups"] = _log(rng, 1, 24)
    c["heads"] = c["groups"] * rng.choice([1, 1, 1, 2, 4])
    if op == "step":
        c["batch"] = _log(rng, 1, 64)
        return c
    c["docs"] = rng.choice([1, 1, 2, 6])
    c["init"] = rng.random() < 0.5
    tokens = 40 * 8192 // max(8, c["heads"])
    c["seqlen"] = _log(rng, 1, min(8192, tokens))
    c["batch"] = _log(rng, 1, max(1, min(8, tokens // c["seqlen"])))
    return c


def _shapes(case):
    """The parameters of `blocks` Mamba-2 blocks of model width w: 2 w inner
    channels in heads of 64, a state of 128, conv of 4."""
    w = case["width"]
    inner, heads = 2 * w, max(1, 2 * w // 64)
    conv = inner + 256
    return [(2 * inner + 256 + heads, w), (w, inner), (conv, 4), (conv,), (heads,), (heads,),
            (heads,), (inner,), (w,)] * case["blocks"]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def rnd(*shape, by=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * by

    def uni(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=dict(case))
    if case["op"] != "adamw":
        t, K, V = DT[case["dtype"]], case["dstate"], case["headdim"]
        G, H, B = case["groups"], case["heads"], case["batch"]
        lead = (B,) if case["op"] == "step" else (B, case["seqlen"])
        unit = torch.nn.functional.normalize
        # v is a slice of the convolved projection (q | k | v); q and k were normalised
        conv = rnd(*lead, 2 * G * K + H * V).to(t)
        rate = torch.exp(uni(H) * math.log(16.0))              # A in 1 .. 16
        dt = torch.exp(uni(*lead, H) * math.log(100.0) - math.log(1000.0))
        s.update(q=unit(rnd(*lead, G, K), dim=-1).to(t), k=unit(rnd(*lead, G, K), dim=-1).to(t),
                 v=conv[..., 2 * G * K:].unflatten(-1, (H, V)), g=-rate * dt,
                 beta=torch.sigmoid(rnd(*lead, H)))
        if case["op"] == "step":
            s.update(v=s["v"].contiguous(), state=rnd(B, H, V, K, by=0.2))
            return s
        if case["init"]:
            s.update(init=rnd(B, H, V, K, by=0.2))
        if case["docs"] > 1:
            cut = uni(B, case["docs"] - 1) * case["seqlen"]
            pos = torch.arange(case["seqlen"], device="cuda")
            s.update(seq=(pos[None, :, None] >= cut[:, None, :]).sum(-1).to(torch.int32))
        if case["op"] == "train":
            s.update(dout=rnd(*lead, H, V).to(t))
        return s
    sizes = [math.prod(v) for v in _shapes(case)]
    n = sum(sizes)

    def split(flat):
        return [v.view(shape) for v, shape in zip(flat.split(sizes), _shapes(case))]

    master = rnd(n, by=0.02)
    s.update(step=1000 + seed % 1000, lr=3e-4, seed=seed % 65536, grad=rnd(n, by=1e-3).to(DT[case["grad"]]))
    if case["param"] == "bf16":
        s.update(param=master.to(torch.bfloat16), master=master)
    else:
        s.update(param=master, master=None)
    state = dict(master=None if s["master"] is None else split(master))
    if case["bits"] == 32:
        s.update(m=rnd(n, by=3e-4), v=uni(n) * 2e-6 + 1e-8)
        state.update(exp_avg=split(s["m"]), exp_avg_sq=split(s["v"]))
    else:
        blocks = [-(-k // BLOCK) for k in sizes]
        first = torch.tensor([0] + blocks[:-1], device="cuda").cumsum(0) * BLOCK
        start = torch.tensor([0] + sizes[:-1], device="cuda").cumsum(0)
        size = torch.tensor(sizes, device="cuda")
        # where each value stands in a layout of whole blocks, and its tensor and place there
        s.update(of=torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), size,
                                            output_size=n))
        s.update(place=torch.arange(n, device="cuda") - start[s["of"]])
        s.update(at=first[s["of"]] + s["place"], blocks=sum(blocks))
        s.update(m=torch.randint(-127, 128, (n,), generator=g, device="cuda").to(torch.int8),
                 v=torch.randint(1, 256, (n,), generator=g, device="cuda").to(torch.uint8),
                 m_scale=1e-3 * (0.5 + uni(sum(blocks))), v_scale=3e-6 * (0.5 + uni(sum(blocks))),
                 m_value=torch.empty(n, device="cuda"), v_value=torch.empty(n, device="cuda"))
        state.update(exp_avg=split(s["m"]), exp_avg_sq=split(s["v"]),
                     exp_avg_scale=list(s["m_scale"].split(blocks)),
                     exp_avg_sq_scale=list(s["v_scale"].split(blocks)))
        s.update(values=(split(s["m_value"]), split(s["v_value"])))
    norm = s["grad"].float().square().sum().sqrt()
    s.update(norm=norm, max_norm=0.5e-3 * n ** 0.5, state=state, params=split(s["param"]),
             grads=split(s["grad"]))
    return s


# ------------------------------------------------------------ plain forms

def _heads(t, H):
    """[B, L, groups, n] -> [B, H, L, n] in fp32, a group's row for each of its heads."""
    return t.float().repeat_interleave(H // t.shape[-2], -2).transpose(1, 2)


def _chunks(t):
    """[B, H, L, ...] -> [B, H, chunks, CHUNK, ...], zeros behind the last token."""
    pad = -t.shape[2] % CHUNK
    if pad:
        t = torch.cat([t, t.new_zeros(t.shape[:2] + (pad,) + t.shape[3:])], 2)
    return t.unflatten(2, (-1, CHUNK))


def _inverse(a):
    """(I + a)^-1 of strictly lower triangular a, by the finite product
    (I - a)(I + a^2)(I + a^4)..."""
    eye = torch.eye(CHUNK, device=a.device)
    inv, p, n = eye - a, a, 2
    while n < CHUNK:
        p = p @ p
        inv = inv + inv @ p
        n *= 2
    return inv


def _delta_parts(s):
    """What the chunks' products need and no state: q, k, v and the decays
    within each chunk."""
    c = s["case"]
    H = c["heads"]
    q, k = (_chunks(_heads(s[n], H)) for n in "qk")
    v = _chunks(s["v"].float().transpose(1, 2))
    beta = _chunks(s["beta"].transpose(1, 2))
    g = _chunks(s["g"].transpose(1, 2).double()).cumsum(-1)
    seg = torch.zeros_like(s["g"][:, :, :1].transpose(1, 2), dtype=torch.int64)
    if "seq" in s:
        q_ = s["seq"]
        new = torch.cat([torch.zeros_like(q_[:, :1]), (q_[:, 1:] != q_[:, :-1]).to(q_.dtype)], 1)
        seg = new.long()[:, None]
    else:
        seg = seg.expand(-1, -1, c["seqlen"])
    seg = _chunks(seg).cumsum(-1)                          # resets up to a token, in its chunk
    tri = torch.ones(CHUNK, CHUNK, device=q.device, dtype=torch.bool).tril()
    near = tri & (seg[..., :, None] == seg[..., None, :])
    decay = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~near, -math.inf)).float()
    into = torch.exp(g.masked_fill(seg != 0, -math.inf)).float()       # from the chunk's start
    last = seg[..., -1:]
    onto = torch.exp((g[..., -1:] - g).masked_fill(seg != last, -math.inf)).float()  # to its end
    through = torch.exp(g[..., -1].masked_fill(last[..., 0] != 0, -math.inf)).float()
    kk = k @ k.transpose(-1, -2)
    qk = q @ k.transpose(-1, -2) * c["dstate"] ** -0.5
    keys = (decay * kk).tril(-1)
    inv = _inverse(keys * beta[..., None, :])
    return dict(q=q * c["dstate"] ** -0.5, k=k, v=v, beta=beta, decay=decay, into=into[..., None],
                onto=onto[..., None], through=through, keys=keys, scores=decay * qk, inv=inv)


def _delta_forward(s, p):
    """The chunks one after another: out, the final state, and each chunk's
    first state and corrections x (u = beta x is what is written)."""
    c = s["case"]
    B, H, V, K = c["batch"], c["heads"], c["headdim"], c["dstate"]
    S = s["init"] if "init" in s else torch.zeros(B, H, V, K, device="cuda")
    states, xs = [], []
    put = p["onto"] * p["beta"][..., None] * p["k"]
    get = p["into"] * p["k"]
    for n in range(p["k"].shape[2]):
        x = p["inv"][:, :, n] @ (p["v"][:, :, n] - get[:, :, n] @ S.transpose(-1, -2))
        states.append(S)
        xs.append(x)
        S = p["through"][:, :, n, None, None] * S + x.transpose(-1, -2) @ put[:, :, n]
    states, x = torch.stack(states, 2), torch.stack(xs, 2)
    o = (p["into"] * p["q"]) @ states.transpose(-1, -2) + p["scores"] @ (p["beta"][..., None] * x)
    return o, S, states, x


def _tokens(t, L):
    """[B, H, chunks, CHUNK, ...] -> [B, L, H, ...]"""
    return t.flatten(2, 3)[:, :, :L].transpose(1, 2)


def _plain_fwd(s):
    c, t = s["case"], s["q"].dtype
    o, S, _, _ = _delta_forward(s, _delta_parts(s))
    return dict(out=_tokens(o, c["seqlen"]).to(t).contiguous(), final_states=S)


def _plain_train(s):
    c, t, L = s["case"], s["q"].dtype, s["case"]["seqlen"]
    p = _delta_parts(s)
    o, _, S0, x = _delta_forward(s, p)
    do = _chunks(s["dout"].float().transpose(1, 2))
    q, k, beta = p["q"], p["k"], p["beta"][..., None]
    put, get, into = p["onto"] * k, p["into"] * k, p["into"]
    dS, dSs, dys = torch.zeros_like(S0[:, :, 0]), [], []
    for n in reversed(range(k.shape[2])):
        dx = beta[:, :, n] * (p["scores"][:, :, n].transpose(-1, -2) @ do[:, :, n]
                              + put[:, :, n] @ dS.transpose(-1, -2))
        dy = p["inv"][:, :, n].transpose(-1, -2) @ dx
        dSs.append(dS)
        dys.append(dy)
        dS = (p["through"][:, :, n, None, None] * dS
              + do[:, :, n].transpose(-1, -2) @ (into * q)[:, :, n]
              - dy.transpose(-1, -2) @ get[:, :, n])
    dSs, dy = torch.stack(dSs[::-1], 2), torch.stack(dys[::-1], 2)
    # gradients through the states: of the reads by q and k, and of the write
    dq0, dk0 = into * (do @ S0), -into * (dy @ S0)
    dw0 = p["onto"] * (x @ dSs)
    # through the pairs of a chunk
    ds = (do @ x.transpose(-1, -2)) * p["decay"]
    dn = -(dy @ x.transpose(-1, -2)) * p["decay"].tril(-1)
    b = p["beta"][..., None, :]
    scale = c["dstate"] ** -0.5
    dq = scale * (dq0 + (ds * b) @ k)
    w = dw0 + ds.transpose(-1, -2) @ q + dn.transpose(-1, -2) @ k
    dk = dk0 + (dn * b) @ k + beta * w
    # the decay of token t is part of every pair around it
    pair = b * ((do @ x.transpose(-1, -2)) * p["scores"] - (dy @ x.transpose(-1, -2)) * p["keys"])
    read = ((q * dq0) + (k * dk0)).sum(-1)
    write = (beta * k * dw0).sum(-1)
    around = pair.cumsum(-1) - pair                      # keys before t, for each query row
    around = around.flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)
    dg = (read.flip(-1).cumsum(-1).flip(-1) + write.cumsum(-1) - write + around
          + (p["through"] * (dSs * S0).sum((-1, -2)))[..., None])
    if "seq" in s:                                       # a reset's own decay has no effect
        new = torch.cat([torch.zeros_like(s["seq"][:, :1], dtype=torch.bool),
                         s["seq"][:, 1:] != s["seq"][:, :-1]], 1)
        dg = dg.masked_fill(_chunks(new[:, None]), 0.0)
    r = c["heads"] // c["groups"]

    def group(v):
        return _tokens(v, L).unflatten(2, (-1, r)).sum(3).to(t)

    out = dict(out=_tokens(o, L).to(t).contiguous(), dq=group(dq), dk=group(dk),
               dv=_tokens(dy, L).to(t).contiguous(), dg=_tokens(dg, L).contiguous(),
               dbeta=_tokens((k * w).sum(-1), L).contiguous())
    if "init" in s:
        out.update(d_initial_states=dS)
    return out


def _plain_step(s):
    c, t = s["case"], s["q"].dtype
    r = c["heads"] // c["groups"]
    q, k = (s[n].float().repeat_interleave(r, 1) for n in "qk")
    S = s["state"]
    S.mul_(torch.exp(s["g"])[..., None, None])
    u = s["beta"][..., None] * (s["v"].float() - (S * k[:, :, None]).sum(-1))
    S.add_(u[..., None] * k[:, :, None])
    return dict(out=((S * q[:, :, None]).sum(-1) * c["dstate"] ** -0.5).to(t), state=S)


def _uniform(s):
    """Two numbers in (0, 1) for each value, of 16 bits each: a mix of the
    seed, the step, the tensor's number and the value's place in it."""
    low = 0xFFFFFFFF

    def mix(h):
        h = ((h ^ (h >> 16)) * 0x7FEB352D) & low
        h = ((h ^ (h >> 15)) * 0x846CA68B) & low
        return h ^ (h >> 16)

    key = mix(torch.tensor(s["seed"], device="cuda"))
    key = mix((key + s["step"]) & low)
    key = mix((key + s["of"]) & low)
    h = mix((key + s["place"]) & low)      # places are below 2^32 here
    return (((h >> 16).float() + 0.5) * 2.0 ** -16, ((h & 0xFFFF).float() + 0.5) * 2.0 ** -16)


def _values(s):
    """The 8-bit moments' values."""
    blk = s["at"] // BLOCK
    t = s["m"].float() * torch.tensor(1.0 / 127.0, device="cuda")
    u = s["v"].float() * torch.tensor(1.0 / 255.0, device="cuda")
    u = u * u
    return (t * t.abs()) * s["m_scale"][blk], (u * u) * s["v_scale"][blk]


def _encode(x, root, top, u, s):
    """Codes of x >= 0 whose value is (code / top)^root of their block's
    largest, up or down with the odds that keep the mean; and the scales."""
    full = torch.zeros(s["blocks"] * BLOCK, device="cuda")
    full[s["at"]] = x
    big = full.view(-1, BLOCK).amax(1)
    r = x / big[s["at"] // BLOCK]
    r = torch.where(x > 0, r, torch.zeros_like(r))
    y = torch.sqrt(r) if root == 2 else torch.sqrt(torch.sqrt(r))
    c = torch.clamp(torch.floor(y * top), max=top - 1.0)
    step = torch.tensor(1.0 / top, device="cuda")
    lo, hi = c * step, (c + 1.0) * step
    lo, hi = lo * lo, hi * hi
    if root == 4:
        lo, hi = lo * lo, hi * hi
    c = c + (u < (r - lo) / (hi - lo)).float()
    return c, big


def _plain_adamw(s):
    (b1, b2), step = BETAS, s["step"]
    g = s["grad"].float()
    if s["case"]["clip"]:
        g = g * torch.clamp(s["max_norm"] / (s["norm"] + 1e-6), max=1.0)
    bits8 = s["case"]["bits"] == 8
    m, v = _values(s) if bits8 else (s["m"], s["v"])
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    p = s["param"] if s["master"] is None else s["master"]
    denom = torch.sqrt(v) * (1.0 / math.sqrt(1.0 - b2 ** step)) + EPS
    p.copy_(p * (1.0 - s["lr"] * DECAY) - m * (s["lr"] / (1.0 - b1 ** step)) / denom)
    if s["master"] is not None:
        s["param"].copy_(p)
    if bits8:
        um, uv = _uniform(s)
        c, big = _encode(m.abs(), 2, 127.0, um, s)
        s["m"].copy_(c * torch.sign(m))
        s["m_scale"].copy_(big)
        c, big = _encode(v, 4, 255.0, uv, s)
        s["v"].copy_(torch.where(v > 0, torch.clamp(c, min=1.0), c))
        s["v_scale"].copy_(big)
        m, v = _values(s)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return dict(param=s["param"], master=s["master"], exp_avg=m if bits8 else s["m"],
                exp_avg_sq=v if bits8 else s["v"])


# ------------------------------------------------------------ the framework's calls

def _own(s):
    import selective_state_space_05_gb300 as ssd
    op = s["case"]["op"]
    if op == "step":
        out = ssd.delta_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"])
        return dict(out=out, state=s["state"])
    if op == "adamw":
        clip = dict(grad_norm=s["norm"], max_norm=s["max_norm"]) if s["case"]["clip"] else {}
        ssd.adamw_step(s["params"], s["grads"], s["state"], step=s["step"], lr=s["lr"], betas=BETAS,
                       eps=EPS, weight_decay=DECAY, seed=s["seed"], **clip)
        o = dict(param=s["param"], master=s["master"])
        if s["case"]["bits"] == 8:
            ssd.adamw_moments(s["state"], out=s["values"])
            return dict(o, exp_avg=s["m_value"], exp_avg_sq=s["v_value"])
        return dict(o, exp_avg=s["m"], exp_avg_sq=s["v"])
    ins = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    kw = dict(initial_states=s.get("init"), seq_idx=s.get("seq"))
    if op == "fwd":
        out, final = ssd.delta_scan_fwd(*ins, return_final_states=True, **kw)
        return dict(out=out, final_states=final)
    out, saved = ssd.delta_scan_fwd(*ins, save=True, **kw)
    grads = ssd.delta_scan_bwd(s["dout"], *ins, saved=saved, **kw)
    return dict({k: v for k, v in grads.items() if v is not None}, out=out)


PLAIN = {"step": _plain_step, "fwd": _plain_fwd, "train": _plain_train, "adamw": _plain_adamw}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(v) for v in _shapes(case))
        b = (2 if case["grad"] == "bf16" else 4) + (10 if case["param"] == "bf16" else 8)
        # moments in and out; those of 8 bits also out as the values they stand for
        b += 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
        return dict(bytes=n * b, flops=n * (15 if case["bits"] == 32 else 50))
    e = 2 if case["dtype"] == "bf16" else 4
    K, V, H, G = case["dstate"], case["headdim"], case["heads"], case["groups"]
    if case["op"] == "step":
        n = case["batch"]
        return dict(bytes=n * (2 * G * K * e + 2 * H * V * e + 8 * H + 8 * H * V * K),
                    flops=n * H * (7 * V * K))
    n = case["batch"] * case["seqlen"]
    states = case["batch"] * H * V * K * 4
    docs = 4 * n if case["docs"] > 1 else 0
    b = n * (2 * G * K * e + 2 * H * V * e + 8 * H) + docs
    # the recurrence's own products: S k, S q and the write, 2 V K each
    f = n * H * 6 * V * K
    if case["op"] == "fwd":
        return dict(bytes=b + states * (2 if case["init"] else 1), flops=f)
    # dout in; dq, dk, dv, dg, dbeta out; the states' gradients take twice the forward's products
    b += n * (2 * G * K * e + 2 * H * V * e + 8 * H) + (2 * states if case["init"] else 0)
    return dict(bytes=b, flops=3 * f)


# ------------------------------------------------------------ the definitions in 64 bits

def _recur(S, q, k, v, g, beta, keep):
    """Token by token: S [B, H, V, K], the others [B, L, H, ...] in 64 bits,
    keep [B, L]: 0 where a document starts."""
    outs = []
    for t in range(q.shape[1]):
        S = S * (torch.exp(g[:, t]) * keep[:, t, None])[..., None, None]
        err = v[:, t] - (S @ k[:, t, :, :, None])[..., 0]
        S = S + (beta[:, t, :, None] * err)[..., None] * k[:, t, :, None]
        outs.append((S @ q[:, t, :, :, None])[..., 0])
    return torch.stack(outs, 1), S


def _exact_delta(s):
    c = s["case"]
    L, r, scale = c["seqlen"], c["heads"] // c["groups"], c["dstate"] ** -0.5
    S = s["init"].double() if "init" in s else torch.zeros(
        c["batch"], c["heads"], c["headdim"], c["dstate"], device="cuda", dtype=torch.float64)
    keep = torch.ones(c["batch"], L, device="cuda", dtype=torch.float64)
    if "seq" in s:
        keep[:, 1:] = (s["seq"][:, 1:] == s["seq"][:, :-1]).double()
    names = ("q", "k", "v", "g", "beta")
    part = 64

    def piece(a):
        got = [s[n][:, a:a + part].double() for n in names]
        if c["op"] == "train":
            got = [t.requires_grad_(True) for t in got]
        q, k = (t.repeat_interleave(r, 2) for t in got[:2])
        return got, (q * scale, k, *got[2:], keep[:, a:a + part])

    outs, firsts = [], []
    for a in range(0, L, part):
        firsts.append(S)
        with torch.no_grad():
            o, S = _recur(S, *piece(a)[1])
        outs.append(o)
    res = dict(out=torch.cat(outs, 1))
    if c["op"] == "fwd":
        return dict(res, final_states=S)
    dS, grads = torch.zeros_like(S), []
    for a, first in reversed(list(zip(range(0, L, part), firsts))):
        leaves, args = piece(a)
        first = first.detach().requires_grad_(True)
        o, S = _recur(first, *args)
        *gr, dS = torch.autograd.grad((o, S), leaves + [first],
                                      (s["dout"][:, a:a + part].double(), dS))
        grads.append(gr)
    for i, n in enumerate(names):
        res["d" + n] = torch.cat([gr[i] for gr in reversed(grads)], 1)
    if "init" in s:
        res.update(d_initial_states=dS)
    return res


def exact(case, seed):
    """The recurrence token by token in 64 bits, its gradients by automatic
    differentiation; the optimizer's update in 64 bits (moments of 8 bits are
    rounded values: they have no counterpart there)."""
    s = prepare(case, seed)
    if case["op"] == "step":
        s.update(case=dict(case, seqlen=1, docs=1, op="fwd"), init=s["state"])
        s.update({n: s[n][:, None] for n in ("q", "k", "v", "g", "beta")})
        o = _exact_delta(s)
        return dict(out=o["out"][:, 0], state=o["final_states"])
    if case["op"] != "adamw":
        return _exact_delta(s)
    (b1, b2), g = BETAS, s["grad"].double()
    if case["clip"]:
        g = g * min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
    if case["bits"] == 8:
        m = s["m"].double() / 127
        blk = s["at"] // BLOCK
        m = m * m.abs() * s["m_scale"].double()[blk]
        v = (s["v"].double() / 255) ** 4 * s["v_scale"].double()[blk]
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = (s["param"] if s["master"] is None else s["master"]).double()
    hat_m, hat_v = m / (1 - b1 ** s["step"]), v / (1 - b2 ** s["step"])
    p = p - s["lr"] * DECAY * p - s["lr"] * hat_m / (hat_v.sqrt() + EPS)
    whole = case["bits"] == 32
    return dict(param=p, master=None if s["master"] is None else p, exp_avg=m if whole else None,
                exp_avg_sq=v if whole else None)
