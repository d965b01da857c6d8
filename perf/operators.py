"""The operators that surround and extend the attention in a decoder block, as measured cases.

  rope   rotary positions for the heads of a qkv product, forward and backward
  norm   RMS norm of rows, and the join of a residual stream with a branch (norm after the branch,
         gate, residual scale, norm before the next branch), forward and training
  diff   differential attention (the difference of two softmax maps), forward and training

``run`` computes a case in its plain form with elementary torch operations in 32 bits (angles in 64),
or, where ``own`` is set, through this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


# ----------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a token of a long generation: only the call's latency counts; scaled for a long context
        dict(name="rope one token", op="rope", dir="fwd", B=1, S=1, H=32, Hkv=8, D=128, rot=128,
             layout="half", dtype="bf16", positions="start", start=131071, factor=4.0),
        # the decoder block's own shape over a training batch, straight from the qkv product
        dict(name="rope training batch", op="rope", dir="fwd", B=2, S=8192, H=32, Hkv=8, D=128,
             rot=128, layout="half", dtype="bf16", positions="start", start=0, factor=1.0),
        # gradients of a part of the head, interleaved pairs, positions of packed documents, 32 bits
        dict(name="rope backward part of head", op="rope", dir="bwd", B=3, S=1237, H=16, Hkv=4, D=64,
             rot=32, layout="interleaved", dtype="fp32", positions="given", start=0, factor=1.0),
        # a token of a generation through the residual stream
        dict(name="join one token", op="join", dir="fwd", B=1, S=1, C=4096, gate="channel",
             dtype="bf16"),
        # the residual stream of a long prefill
        dict(name="join forward", op="join", dir="fwd", B=2, S=8192, C=4096, gate="channel",
             dtype="bf16"),
        # a training step whose gate is conditioned on the sequence
        dict(name="join training", op="join", dir="train", B=4, S=4096, C=4096, gate="sequence",
             dtype="bf16"),
        # an odd width and length, 32 bits
        dict(name="norm training odd", op="norm", dir="train", B=3, S=1237, C=1001, dtype="fp32"),
        # the norm of every head of an attention output
        dict(name="norm of heads training", op="norm", dir="train", B=16, S=32768, C=128,
             dtype="bf16"),
        # a short prompt
        dict(name="diff short forward", op="diff", dir="fwd", B=1, S=17, H=4, Hkv=2, d=64,
             causal=True, lam="head"),
        # a long prefill at the decoder block's shape
        dict(name="diff forward", op="diff", dir="fwd", B=1, S=8192, H=32, Hkv=8, d=64, causal=True,
             lam="head"),
        # a training step of the same
        dict(name="diff training", op="diff", dir="train", B=1, S=8192, H=32, Hkv=8, d=64,
             causal=True, lam="head"),
        # smaller heads, no mask, a weight for every token, a ragged length
        dict(name="diff training ragged", op="diff", dir="train", B=3, S=1237, H=16, Hkv=16, d=32,
             causal=False, lam="token"),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "join", "norm", "diff"])
    if op == "rope":
        D = rng.choice([32, 64, 96, 128, 256])
        Hkv = rng.randint(1, 8)
        H = Hkv * rng.randint(1, 4)
        B = rng.randint(1, 4)
        S = _log(rng, 1, max(2, 2 ** 25 // (B * (H + 2 * Hkv) * D)))
        return dict(op="rope", dir=rng.choice(["fwd", "bwd"]), B=B, S=S, H=H, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2]), layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    positions=rng.choice(["start", "given"]), start=rng.randint(0, 1 << 20),
                    factor=rng.choice([1.0, 4.0, 32.0]))
    if op in ("join", "norm"):
        C = rng.choice([_log(rng, 64, 16384), 64 * _log(rng, 1, 256)])
        B = rng.randint(1, 4)
        S = _log(rng, 1, max(2, 2 ** 25 // (B * C)))
        case = dict(op=op, dir=rng.choice(["fwd", "train"]), B=B, S=S, C=C,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        if op == "join":
            case["gate"] = rng.choice(["none", "channel", "sequence"])
        return case
    d = rng.choice([32, 64])
    Hkv = rng.randint(1, 8)
    H = Hkv * rng.randint(1, 4)
    B = rng.randint(1, 3)
    direction = rng.choice(["fwd", "train"])
    return dict(op="diff", dir=direction, B=B, S=_log(rng, 1 if direction == "fwd" else 40, 4096),
                H=H, Hkv=Hkv, d=d, causal=rng.random() < 0.5, lam=rng.choice(["head", "token"]))


# ---------------------------------------------------------------------------------- the inputs
def _frequencies(case):
    """Radians per position of each pair, 64 bits: base 10000, slowed by `factor` from the pair
    that turns less than once over the first 4096 positions on, kept where a pair turns 32 times,
    with a ramp over the pairs in between."""
    n = case["rot"] // 2
    f = torch.tensor([10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64)
    if case["factor"] == 1.0:
        return f, 1.0
    turns = f * 4096.0 / (2.0 * math.pi)
    pair = torch.arange(n, dtype=torch.float64)
    first = float((turns > 32.0).sum())
    last = max(first + 1.0, float((turns > 1.0).sum()))
    keep = 1.0 - ((pair - first) / (last - first)).clamp(0.0, 1.0)
    return f * keep + f / case["factor"] * (1.0 - keep), 0.1 * math.log(case["factor"]) + 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, by=1.0, plus=0.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(by).add_(plus).to(dtype)

    B, S = case["B"], case["S"]
    st = dict(case=dict(case))
    if case["op"] == "rope":
        dt, D, H, Hkv = DTYPES[case["dtype"]], case["D"], case["H"], case["Hkv"]
        f, st["magnitude"] = _frequencies(case)
        st["inv_freq"] = f.cuda()
        if case["positions"] == "given":  # documents that begin anywhere: positions rise from each start
            begin = torch.randint(0, 1 << 17, (B, 1), generator=g, device="cuda")
            st["positions"] = begin + torch.arange(S, device="cuda")
        else:
            st["positions"] = None
        if case["dir"] == "fwd":  # heads as views of one qkv product
            qkv = randn(B, S, (H + 2 * Hkv) * D, dtype=dt)
            parts = qkv.split([H * D, Hkv * D, Hkv * D], dim=-1)
            st["parts"] = tuple(p.unflatten(-1, (-1, D)) for p in parts)
        else:  # gradients as the attention backward leaves them
            st["parts"] = tuple(randn(B, S, h, D, dtype=dt) for h in (H, Hkv, Hkv))
    elif case["op"] in ("join", "norm"):
        dt, C = DTYPES[case["dtype"]], case["C"]
        st["x"] = randn(B, S, C, dtype=dt, by=2.0)
        st["w_next"] = randn(C, dtype=dt, by=0.1, plus=1.0)
        if case["op"] == "join":
            st["a"] = randn(B, S, C, dtype=dt, by=0.5)
            st["w_post"] = randn(C, dtype=dt, by=0.1, plus=1.0)
            shape = {"none": None, "channel": (C,), "sequence": (B, C)}[case["gate"]]
            st["gate"] = None if shape is None else randn(*shape, dtype=dt, by=0.3, plus=0.5)
        if case["dir"] == "train":
            st["dh"] = randn(B, S, C, dtype=dt)
            if case["op"] == "join":
                st["dy"] = randn(B, S, C, dtype=dt)
    else:
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        # scores of trained heads spread over several units
        st["q"] = randn(B, S, 2 * H, d, by=2.0)
        st["k"] = randn(B, S, 2 * Hkv, d)
        st["v"] = randn(B, S, Hkv, 2 * d)
        shape = (H,) if case["lam"] == "head" else (B, S, H)
        lam = torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)
        st["lam"] = (0.2 + 0.6 * lam).to(torch.bfloat16)
        if case["dir"] == "train":
            st["do"] = randn(B, S, H, 2 * d)
    return st


# ---------------------------------------------------------------------------------- one pass
SKIP, BRANCH = 1.0, 0.7  # residual scales of the join


def run(st):
    return {"rope": _rope, "join": _join, "norm": _norm, "diff": _diff}[st["case"]["op"]](st)


def _rope(st):
    c = st["case"]
    B, S, D, back = c["B"], c["S"], c["D"], c["dir"] == "bwd"
    if own:
        import deterministic_attention_backward_gb300 as dash
        args = dict(inv_freq=st["inv_freq"], magnitude=st["magnitude"], positions=st["positions"],
                    start=c["start"], layout=c["layout"])
        if not back:
            return dash.rope_fwd(*st["parts"], **args)
        widths = [p.shape[2] * D for p in st["parts"]]
        dqkv = torch.empty(B, S, sum(widths), dtype=st["parts"][0].dtype, device="cuda")
        out = tuple(p.unflatten(-1, (-1, D)) for p in dqkv.split(widths, dim=-1))
        dash.rope_bwd(*st["parts"], out=out, **args)
        return dqkv
    pos = st["positions"]
    if pos is None:
        pos = (c["start"] + torch.arange(S, device="cuda")).expand(B, S)
    angle = pos.double()[..., None, None] * st["inv_freq"]
    cos = (angle.cos() * st["magnitude"]).float()
    sin = (angle.sin() * (-st["magnitude"] if back else st["magnitude"])).float()

    def turn(x):
        y = x.float()
        rot, rest = y[..., : c["rot"]], y[..., c["rot"]:]
        if c["layout"] == "half":
            a, b = rot.chunk(2, dim=-1)
            rot = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([rot, rest], dim=-1).to(x.dtype)

    q, k, v = st["parts"]
    q, k, v = turn(q), turn(k), v.contiguous()
    if not back:
        return q, k, v
    return torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], dim=-1)


def _rms_grad(g, xhat, rstd):
    return rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))


def _norm(st):
    x, w = st["x"], st["w_next"]
    train = st["case"]["dir"] == "train"
    if own:
        import deterministic_attention_backward_gb300 as dash
        h, rstd = dash.norm_fwd(x, w, eps=EPS)
        if not train:
            return dict(h=h)
        dx, dw = dash.norm_bwd(st["dh"], x, rstd, w)
        return dict(h=h, dx=dx, dw=dw)
    xf, wf = x.float(), w.float()
    rstd = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    xhat = xf * rstd
    out = dict(h=(xhat * wf).to(x.dtype))
    if train:
        dh = st["dh"].float()
        out["dx"] = _rms_grad(dh * wf, xhat, rstd).to(x.dtype)
        out["dw"] = (dh * xhat).sum((0, 1)).to(w.dtype)
    return out


def _join(st):
    x, a, gate = st["x"], st["a"], st["gate"]
    train = st["case"]["dir"] == "train"
    if own:
        import deterministic_attention_backward_gb300 as dash
        weights = dict(w_post=st["w_post"], gate=gate, w_next=st["w_next"])
        scales = dict(skip_scale=SKIP, branch_scale=BRANCH)
        y, h, rstd_a, rstd_y = dash.join_fwd(x, a, **weights, **scales, eps=EPS)
        if not train:
            return dict(y=y, h=h)
        dx, da, dw_post, dgate, dw_next = dash.join_bwd(st["dy"], st["dh"], y, a, rstd_a, rstd_y,
                                                        **weights, **scales)
        out = dict(y=y, h=h, dx=dx, da=da, dw_post=dw_post, dw_next=dw_next)
        return out if gate is None else dict(out, dgate=dgate)
    xf, af, wp, wn = x.float(), a.float(), st["w_post"].float(), st["w_next"].float()
    g = torch.ones((), device="cuda") if gate is None else gate.float()
    g = g[:, None, :] if g.dim() == 2 else g
    rstd_a = torch.rsqrt(af.square().mean(-1, keepdim=True) + EPS)
    ahat = af * rstd_a
    y = SKIP * xf + BRANCH * g * (ahat * wp)
    rstd_y = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    yhat = y * rstd_y
    out = dict(y=y.to(x.dtype), h=(yhat * wn).to(x.dtype))
    if not train:
        return out
    dh = st["dh"].float()
    dy = st["dy"].float() + _rms_grad(dh * wn, yhat, rstd_y)
    dz = BRANCH * g * dy
    out["dx"] = (SKIP * dy).to(x.dtype)
    out["da"] = _rms_grad(dz * wp, ahat, rstd_a).to(x.dtype)
    out["dw_post"] = (dz * ahat).sum((0, 1)).to(x.dtype)
    out["dw_next"] = (dh * yhat).sum((0, 1)).to(x.dtype)
    if gate is not None:
        dg = BRANCH * dy * ahat * wp
        out["dgate"] = dg.sum((0, 1) if gate.dim() == 1 else 1).to(x.dtype)
    return out


def _diff(st):
    c = st["case"]
    q, k, v, lam = st["q"], st["k"], st["v"], st["lam"]
    train = c["dir"] == "train"
    if own:
        import deterministic_attention_backward_gb300 as dash
        o, o2, lse = dash.diff_fwd(q, k, v, lam, causal=c["causal"])
        if not train:
            return dict(o=o, o2=o2, lse=lse)
        dq, dk, dv, dlam = dash.diff_bwd(q, k, v, o, o2, st["do"], lse, lam, causal=c["causal"])
        return dict(o=o, dq=dq, dk=dk, dv=dv, dlam=dlam)
    B, S, H, Hkv, d = c["B"], c["S"], c["H"], c["Hkv"], c["d"]
    G, scale = H // Hkv, c["d"] ** -0.5
    # maps as a leading axis: [2, B, H, S, d]; key and value heads repeated for their query heads
    qf = q.float().view(B, S, H, 2, d).permute(3, 0, 2, 1, 4)
    kf = k.float().view(B, S, Hkv, 2, d).permute(3, 0, 2, 1, 4).repeat_interleave(G, dim=2)
    vf = v.float().transpose(1, 2).repeat_interleave(G, dim=1)
    s = (qf @ kf.transpose(-1, -2)).mul_(scale)
    if c["causal"]:
        at = torch.arange(S, device="cuda")
        s.masked_fill_(at[None, :] > at[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total)
    lse = (top + total.log()).squeeze(-1)
    each = p @ vf
    lf = lam.float()
    lf = lf[None, :, None, None] if lf.dim() == 1 else lf.transpose(1, 2)[..., None]
    o = (each[0] - lf * each[1]).transpose(1, 2).to(q.dtype)
    if not train:
        return dict(o=o, o2=each[1].transpose(1, 2).to(q.dtype),
                    lse=lse.permute(1, 2, 0, 3).reshape(B, 2 * H, S))
    do = st["do"].float().transpose(1, 2)
    dp = do @ vf.transpose(-1, -2)
    delta = (do * each).sum(-1, keepdim=True)
    dlam = -delta[1].squeeze(-1)
    dlam = dlam.sum((0, 2)) if lam.dim() == 1 else dlam.transpose(1, 2)
    dv = ((p[0] - lf * p[1]).transpose(-1, -2) @ do)
    ds = p.mul_(dp - delta).mul_(scale)
    ds[1].mul_(-lf)
    dq = ds @ kf
    dk = ds.transpose(-1, -2) @ qf

    def shared(t):  # sum over the query heads of a key and value head
        return t.unflatten(-3, (Hkv, G)).sum(-3)

    return dict(o=o, dq=dq.permute(1, 3, 2, 0, 4).reshape(B, S, 2 * H, d).to(q.dtype),
                dk=shared(dk).permute(1, 3, 2, 0, 4).reshape(B, S, 2 * Hkv, d).to(q.dtype),
                dv=shared(dv).transpose(1, 2).to(q.dtype), dlam=dlam.to(lam.dtype))


# --------------------------------------------------------------------- what a pass cannot do without
def work(case):
    B, S = case["B"], case["S"]
    e = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("dtype", "bf16")]
    if case["op"] == "rope":
        heads = case["H"] + 2 * case["Hkv"]
        pos = 8 * B * S if case["positions"] == "given" else 0
        return dict(bytes=2 * B * S * heads * case["D"] * e + pos,
                    flops=3 * B * S * (case["H"] + case["Hkv"]) * case["rot"])
    if case["op"] in ("join", "norm"):
        n, C, join, train = B * S * case["C"], case["C"], case["op"] == "join", case["dir"] == "train"
        # forward: x (and a) in, h (and y) out; backward: dh, the normed rows (and dy, a) in, dx (and da) out
        moved = (4 if join else 2) + ((6 if join else 3) if train else 0)
        weights = (4 if join else 1) * C * e * (3 if train else 1)
        return dict(bytes=moved * n * e + weights, flops=((12 if join else 4) + ((22 if join else 9) if train else 0)) * n)
    H, Hkv, d, train = case["H"], case["Hkv"], case["d"], case["dir"] == "train"
    dv = 2 * d
    pairs = B * H * (S * (S + 1) // 2 if case["causal"] else S * S)
    rows = 2 * B * S
    # forward: q, k, v in, o, o2, lse out; backward: those and do in, dq, dk, dv out
    fwd = rows * (2 * H * d + 2 * Hkv * d + Hkv * dv + 2 * H * dv) + 8 * B * S * H
    bwd = rows * (4 * H * d + 4 * Hkv * d + 2 * Hkv * dv + 3 * H * dv) + 8 * B * S * H
    return dict(bytes=fwd + (bwd if train else 0),
                flops=pairs * 2 * ((2 * d + 2 * dv) + ((6 * d + 2 * dv) if train else 0)))


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "join": _exact_rows, "norm": _exact_rows, "diff": _exact_diff}[case["op"]](case, st)


def _exact_rope(case, st):
    """Each pair as a complex number, turned by exp(i angle)."""
    B, S, n = case["B"], case["S"], case["rot"] // 2
    pos = st["positions"]
    if pos is None:
        pos = torch.full((B, S), case["start"], device="cuda") + torch.arange(S, device="cuda")
    sign = -1.0 if case["dir"] == "bwd" else 1.0
    by = torch.polar(torch.full((B, S, 1, n), st["magnitude"], dtype=torch.float64, device="cuda"),
                     sign * pos.double()[:, :, None, None] * st["inv_freq"])
    q, k, v = (t.double() for t in st["parts"])
    res = []
    for t in (q, k):
        out = t.clone()
        even = slice(0, n) if case["layout"] == "half" else slice(0, 2 * n, 2)
        odd = slice(n, 2 * n) if case["layout"] == "half" else slice(1, 2 * n, 2)
        z = torch.complex(t[..., even].contiguous(), t[..., odd].contiguous()) * by
        out[..., even], out[..., odd] = z.real, z.imag
        res.append(out)
    if case["dir"] == "fwd":
        return res[0], res[1], v
    return torch.cat([t.reshape(B, S, -1) for t in (*res, v)], dim=-1)


def _exact_rows(case, st):
    """The forward's definition, differentiated by autograd."""
    join, train = case["op"] == "join", case["dir"] == "train"
    names = ["x", "w_next"] + (["a", "w_post"] + (["gate"] if st["gate"] is not None else []) if join else [])
    t = {n: st[n].double().requires_grad_(train) for n in names}

    def rms(z, w):
        return z / torch.sqrt((z * z).sum(-1, keepdim=True) / z.shape[-1] + EPS) * w

    if join:
        branch = rms(t["a"], t["w_post"])
        if "gate" in t:
            branch = branch * (t["gate"] if t["gate"].dim() == 1 else t["gate"].unsqueeze(1))
        y = SKIP * t["x"] + BRANCH * branch
        h = rms(y, t["w_next"])
        out = dict(y=y.detach(), h=h.detach())
    else:
        h = rms(t["x"], t["w_next"])
        out = dict(h=h.detach())
    if train:
        loss = (h * st["dh"].double()).sum()
        if join:
            loss = loss + (y * st["dy"].double()).sum()
        grads = dict(zip(names, torch.autograd.grad(loss, [t[n] for n in names])))
        out["dx"] = grads["x"]
        out["dw_next" if join else "dw"] = grads["w_next"]
        if join:
            out["da"], out["dw_post"] = grads["a"], grads["w_post"]
            if "gate" in grads:
                out["dgate"] = grads["gate"]
    return out


def _exact_diff(case, st):
    """One batch entry and query head at a time, each gradient from the chain rule."""
    B, S, H, Hkv, d, train = case["B"], case["S"], case["H"], case["Hkv"], case["d"], case["dir"] == "train"
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, o2, lse = new(B, S, H, 2 * d), new(B, S, H, 2 * d), new(B, 2 * H, S)
    dq, dk, dv = new(B, S, 2 * H, d), new(B, S, 2 * Hkv, d), new(B, S, Hkv, 2 * d)
    dlam = new(*st["lam"].shape)
    hide = torch.ones(S, S, dtype=torch.bool, device="cuda").triu(1) if case["causal"] else None
    for b in range(B):
        for h in range(H):
            n = h // (H // Hkv)
            v = st["v"][b, :, n].double()
            lam = st["lam"].double()
            lam = lam[h] if lam.dim() == 1 else lam[b, :, h][:, None]
            maps = []
            for m in range(2):
                s = st["q"][b, :, 2 * h + m].double() @ st["k"][b, :, 2 * n + m].double().T / math.sqrt(d)
                if hide is not None:
                    s[hide] = -math.inf
                lse[b, 2 * h + m] = torch.logsumexp(s, -1)
                maps.append(torch.softmax(s, -1))
            o2[b, :, h] = maps[1] @ v
            both = maps[0] - lam * maps[1]
            o[b, :, h] = both @ v
            if not train:
                continue
            do = st["do"][b, :, h].double()
            dv[b, :, n] += both.T @ do
            dboth = do @ v.T
            along = (maps[1] * dboth).sum(-1)
            if dlam.dim() == 1:
                dlam[h] -= along.sum()
            else:
                dlam[b, :, h] = -along
            for m in range(2):
                dmap = dboth if m == 0 else -lam * dboth
                ds = maps[m] * (dmap - (maps[m] * dmap).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[b, :, 2 * h + m] = ds @ st["k"][b, :, 2 * n + m].double()
                dk[b, :, 2 * n + m] += ds.T @ st["q"][b, :, 2 * h + m].double()
    if not train:
        return dict(o=o, o2=o2, lse=lse)
    return dict(o=o, dq=dq, dk=dk, dv=dv, dlam=dlam)
