"""The operators that complete a training step of the decoder block, as measured cases.

  heads  RMS norm of every head of q and k with the rotary turn in the same pass, v copied
  dense  matrix product with bias, activation, gate and residual in its epilogue
  clip   the global norm over many gradients, and clipping by it

``run`` computes a case in its plain form with elementary torch operations in 32 bits (angles and the
sum over all gradients in 64), or, where ``own`` is set, through this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


# ----------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a token of a long generation: only the call's latency counts
        dict(name="heads one token", op="heads", dir="fwd", B=1, S=1, H=32, Hkv=8, D=128, rot=128,
             layout="half", dtype="bf16", positions="start", start=131071),
        # a training step at the decoder block's shape, straight from the qkv product and back to it
        dict(name="heads training", op="heads", dir="train", B=2, S=8192, H=32, Hkv=8, D=128,
             rot=128, layout="half", dtype="bf16", positions="start", start=0),
        # a part of the head turned, interleaved pairs, positions of packed documents, 32 bits
        dict(name="heads training part of head", op="heads", dir="train", B=3, S=1237, H=16, Hkv=4,
             D=64, rot=32, layout="interleaved", dtype="fp32", positions="given", start=0),
        # a token of a generation through the block's gated up product
        dict(name="dense one token gated", op="dense", dir="fwd", M=1, K=4096, N=14336, act="silu",
             gate=True, bias=False, residual=False, order="kn", dtype="bf16"),
        # a small batch of sequences that decode together, down product onto the residual stream
        dict(name="dense few tokens", op="dense", dir="fwd", M=17, K=14336, N=4096, act="none",
             gate=False, bias=False, residual=True, order="nk", dtype="bf16"),
        # a long prefill through a product with bias and activation
        dict(name="dense forward", op="dense", dir="fwd", M=8192, K=4096, N=14336, act="gelu",
             gate=False, bias=True, residual=False, order="kn", dtype="bf16"),
        # a training step of the product behind the attention
        dict(name="dense training residual", op="dense", dir="train", M=8192, K=4096, N=4096,
             act="none", gate=False, bias=False, residual=True, order="kn", dtype="bf16"),
        # a training step of the gated up product at the decoder block's shape
        dict(name="dense training gated", op="dense", dir="train", M=8192, K=4096, N=14336,
             act="silu", gate=True, bias=False, residual=False, order="kn", dtype="bf16"),
        # odd sizes, everything in the epilogue, weights stored by outputs
        dict(name="dense training ragged", op="dense", dir="train", M=3711, K=1001, N=777,
             act="gelu_tanh", gate=False, bias=True, residual=True, order="nk", dtype="fp16"),
        # a small model's gradients: many small tensors of odd sizes, nothing to clip
        dict(name="clip small model", op="clip", layers=4, hidden=512, heads=4, kv_heads=2, D=128,
             ffn=777, dtype="bf16", clipped=False),
        # the gradients of one decoder block, clipped
        dict(name="clip block", op="clip", layers=1, hidden=4096, heads=32, kv_heads=8, D=128,
             ffn=14336, dtype="bf16", clipped=True),
        # master gradients in 32 bits of several blocks within the limit, as most steps are
        dict(name="clip several blocks", op="clip", layers=4, hidden=4096, heads=32, kv_heads=8,
             D=128, ffn=14336, dtype="fp32", clipped=False),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["heads", "dense", "dense", "clip"])
    if op == "heads":
        D = rng.choice([32, 64, 96, 128, 256, 80, 50])
        Hkv = rng.randint(1, 8)
        H = Hkv * rng.randint(1, 4)
        B = rng.randint(1, 4)
        S = _log(rng, 1, max(2, 2 ** 25 // (B * (H + 2 * Hkv) * D)))
        return dict(op="heads", dir=rng.choice(["fwd", "train"]), B=B, S=S, H=H, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2 // 2 * 2]), layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    positions=rng.choice(["start", "given"]), start=rng.randint(0, 1 << 20))
    if op == "dense":
        K, N = (rng.choice([_log(rng, 16, 8192), 64 * _log(rng, 1, 128)]) for _ in range(2))
        gate = rng.random() < 0.4
        M = _log(rng, 1, min(8192, int(9e11) // (K * N * (1 + gate))))
        return dict(op="dense", dir=rng.choice(["fwd", "train"]), M=M, K=K, N=N,
                    act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]), gate=gate,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    order=rng.choice(["kn", "nk"]), dtype=rng.choice(["bf16", "bf16", "fp16"]))
    D = rng.choice([32, 64, 128])
    kv_heads = rng.randint(1, 8)
    heads = kv_heads * rng.randint(1, 4)
    hidden, ffn = _log(rng, 30, 4096), _log(rng, 30, 14336)
    size = hidden * ((2 * heads + 2 * kv_heads) * D + 3 * ffn + 2)
    return dict(op="clip", layers=_log(rng, 1, max(1, min(64, (1 << 28) // size))), hidden=hidden,
                heads=heads, kv_heads=kv_heads, D=D, ffn=ffn,
                dtype=rng.choice(["bf16", "fp16", "fp32"]), clipped=rng.random() < 0.5)


# ---------------------------------------------------------------------------------- the inputs
def _gradient_shapes(case):
    h, D = case["hidden"], case["D"]
    block = [(h, (case["heads"] + 2 * case["kv_heads"]) * D), (case["heads"] * D, h),
             (h, case["ffn"]), (h, case["ffn"]), (case["ffn"], h), (h,), (h,)]
    return block * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, by=1.0, plus=0.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(by).add_(plus).to(dtype)

    st = dict(case=dict(case))
    dt = DTYPES[case["dtype"]]
    train = case.get("dir") == "train"
    if case["op"] == "heads":
        B, S, D, H, Hkv = case["B"], case["S"], case["D"], case["H"], case["Hkv"]
        n = case["rot"] // 2
        st["inv_freq"] = torch.tensor([10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64,
                                      device="cuda")
        st["positions"] = None
        if case["positions"] == "given":  # documents that begin anywhere
            begin = torch.randint(0, 1 << 17, (B, 1), generator=g, device="cuda")
            st["positions"] = begin + torch.arange(S, device="cuda")
        # heads as views of one qkv product
        widths = [H * D, Hkv * D, Hkv * D]
        st["parts"] = tuple(p.unflatten(-1, (-1, D)) for p in
                            randn(B, S, sum(widths), dtype=dt, by=2.0).split(widths, dim=-1))
        st["wq"], st["wk"] = (randn(D, dtype=dt, by=0.1, plus=1.0) for _ in range(2))
        if train:  # gradients as the attention backward leaves them
            st["grads"] = tuple(randn(B, S, h, D, dtype=dt) for h in (H, Hkv, Hkv))
    elif case["op"] == "dense":
        M, K, N = case["M"], case["K"], case["N"]

        def weight():
            if case["order"] == "kn":
                return randn(K, N, dtype=dt, by=K ** -0.5)
            return randn(N, K, dtype=dt, by=K ** -0.5).t()
        st["x"], st["w"] = randn(M, K, dtype=dt), weight()
        st["w_gate"] = weight() if case["gate"] else None
        st["bias"] = randn(N, dtype=dt, by=0.2) if case["bias"] else None
        st["bias_gate"] = randn(N, dtype=dt, by=0.2) if case["bias"] and case["gate"] else None
        st["residual"] = randn(M, N, dtype=dt) if case["residual"] else None
        st["dy"] = randn(M, N, dtype=dt) if train else None
    else:
        # each layer's gradients have a size of their own
        st["grads"] = [randn(*s, dtype=dt, by=1e-2 * (1 + i % 5))
                       for i, s in enumerate(_gradient_shapes(case))]
        # the clipped ones go to buffers of an optimizer's; what is not clipped stays in its place
        st["out"] = [torch.empty_like(t) for t in st["grads"]] if case["clipped"] else None
        # the norm is at least 1e-2 sqrt(the number of elements) nearly surely
        count = sum(t.numel() for t in st["grads"])
        st["max_norm"] = (1e-3 if case["clipped"] else 1.0) * math.sqrt(count)
    return st


# ---------------------------------------------------------------------------------- one pass
def run(st):
    return {"heads": _heads, "dense": _dense, "clip": _clip}[st["case"]["op"]](st)


def _heads(st):
    c = st["case"]
    B, S, D, rot, train = c["B"], c["S"], c["D"], c["rot"], c["dir"] == "train"
    wq, wk = st["wq"], st["wk"]
    if own:
        import deterministic_attention_backward_gb300 as dash
        args = dict(q_weight=wq, k_weight=wk, inv_freq=st["inv_freq"], eps=EPS,
                    positions=st["positions"], start=c["start"], layout=c["layout"])
        q, k, v = dash.rope_norm_fwd(*st["parts"], **args)
        if not train:
            return dict(q=q, k=k, v=v)
        widths = [p.shape[2] * D for p in st["parts"]]
        dqkv = torch.empty(B, S, sum(widths), dtype=q.dtype, device="cuda")
        out = tuple(p.unflatten(-1, (-1, D)) for p in dqkv.split(widths, dim=-1))
        *_, dwq, dwk = dash.rope_norm_bwd(*st["grads"], *st["parts"][:2], out=out, **args)
        return dict(q=q, k=k, v=v, dqkv=dqkv, dwq=dwq, dwk=dwk)
    pos = st["positions"]
    if pos is None:
        pos = (c["start"] + torch.arange(S, device="cuda")).expand(B, S)
    angle = pos.double()[..., None, None] * st["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()

    def turn(x, sin):
        front, rest = x[..., :rot], x[..., rot:]
        if c["layout"] == "half":
            a, b = front.chunk(2, dim=-1)
            front = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = front[..., 0::2], front[..., 1::2]
            front = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([front, rest], dim=-1)

    normed, out = [], {}
    for name, x, w in (("q", st["parts"][0], wq), ("k", st["parts"][1], wk)):
        xf = x.float()
        rstd = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
        xhat = xf * rstd
        out[name] = turn(xhat * w.float(), sin).to(x.dtype)
        normed.append((xhat, rstd, w))
    out["v"] = st["parts"][2].contiguous()
    if train:
        grads = []
        for name, dy, (xhat, rstd, w) in zip("qk", st["grads"], normed):
            dz = turn(dy.float(), -sin)
            out["dw" + name] = (dz * xhat).sum((0, 1, 2)).to(w.dtype)
            dz = dz * w.float()
            grads.append(rstd * (dz - xhat * (dz * xhat).mean(-1, keepdim=True)))
        grads.append(st["grads"][2].float())
        out["dqkv"] = torch.cat([t.flatten(2) for t in grads], dim=-1).to(st["parts"][0].dtype)
    return out


def _activation(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0.0), (z > 0.0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * b * z * z)


def _dense(st):
    x, w, wg, act, train = st["x"], st["w"], st["w_gate"], st["case"]["act"], st["dy"] is not None
    if own:
        import deterministic_attention_backward_gb300 as dash
        y, kept = dash.dense_fwd(x, w, st["bias"], act=act, w_gate=wg, bias_gate=st["bias_gate"],
                                 residual=st["residual"], keep=train)
        if not train:
            return dict(y=y)
        dx, dw, db, dwg, dbg = dash.dense_bwd(st["dy"], x, w, kept, act=act, w_gate=wg,
                                              bias=st["bias"], bias_gate=st["bias_gate"])
        out = dict(y=y, dx=dx, dw=dw, db=db, dw_gate=dwg, db_gate=dbg)
        return {n: t for n, t in out.items() if t is not None}
    xf, wf = x.float(), w.float()
    z = xf @ wf
    if st["bias"] is not None:
        z += st["bias"].float()
    y, slope = _activation(z, act)
    if wg is not None:
        gate, plain = xf @ wg.float(), y
        if st["bias_gate"] is not None:
            gate += st["bias_gate"].float()
        y = y * gate
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = dict(y=y.to(x.dtype))
    if not train:
        return out
    dy = st["dy"].float()
    dz = dy * slope
    if wg is not None:
        dz = dz * gate
    dx = dz @ wf.t()
    out["dw"] = (xf.t() @ dz).to(w.dtype)
    if st["bias"] is not None:
        out["db"] = dz.sum(0).to(w.dtype)
    if wg is not None:
        dgate = dy * plain
        dx = dx + dgate @ wg.float().t()
        out["dw_gate"] = (xf.t() @ dgate).to(w.dtype)
        if st["bias_gate"] is not None:
            out["db_gate"] = dgate.sum(0).to(w.dtype)
    out["dx"] = dx.to(x.dtype)
    return out


def _clip(st):
    grads, out = st["grads"], st["out"]
    if own:
        import deterministic_attention_backward_gb300 as dash
        norm = dash.grad_clip(grads, st["max_norm"], out=out)
    else:
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for t in grads:
            total += t.float().square().sum(dtype=torch.float64)
        norm = total.sqrt()
        by = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        norm = norm.float()
        for t, o in zip(grads, grads if out is None else out):
            o.copy_(t.float() * by)
    res = {f"g{i}": t for i, t in enumerate(grads if out is None else out)}
    return dict(res, norm=norm)


# --------------------------------------------------------------------- what a pass cannot do without
def work(case):
    e, train = BYTES[case["dtype"]], case.get("dir") == "train"
    if case["op"] == "heads":
        tokens = case["B"] * case["S"]
        turned = (case["H"] + case["Hkv"]) * case["D"] * tokens
        copied = case["Hkv"] * case["D"] * tokens
        pos = 8 * tokens if case["positions"] == "given" else 0
        # forward: heads in, heads out; backward, a call of its own: their gradients and q and k in,
        # gradients out
        moved = 2 * (turned + copied) + (3 * turned + 2 * copied if train else 0)
        return dict(bytes=moved * e + pos * (2 if train else 1),
                    flops=turned * (7 + (16 if train else 0)))
    if case["op"] == "dense":
        M, K, N, n = case["M"], case["K"], case["N"], 1 + case["gate"]
        moved = M * K + n * K * N + M * N * (1 + case["residual"]) + (n * N if case["bias"] else 0)
        if train:  # dy in; dx and the weights' gradients out
            moved += M * N + M * K + n * K * N + (n * N if case["bias"] else 0)
        return dict(bytes=moved * e, flops=2 * n * M * K * N * (3 if train else 1))
    count = sum(math.prod(s) for s in _gradient_shapes(case))
    # in place, nothing is written where nothing is clipped
    return dict(bytes=count * e * (2 if case["clipped"] else 1), flops=2 * count)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"heads": _exact_heads, "dense": _exact_dense, "clip": _exact_clip}[case["op"]](case, st)


def _exact_heads(case, st):
    """Pairs as complex numbers, turned by exp(i angle); gradients by autograd of the definition."""
    B, S, n, train = case["B"], case["S"], case["rot"] // 2, case["dir"] == "train"
    pos = st["positions"]
    if pos is None:
        pos = torch.full((B, S), case["start"], device="cuda") + torch.arange(S, device="cuda")
    by = torch.polar(torch.ones(B, S, 1, n, dtype=torch.float64, device="cuda"),
                     pos.double()[:, :, None, None] * st["inv_freq"])

    def forward(t, w):
        z = t / torch.sqrt((t * t).sum(-1, keepdim=True) / case["D"] + EPS) * w
        if case["layout"] == "half":
            pair = torch.complex(z[..., :n], z[..., n:2 * n]) * by
            return torch.cat([pair.real, pair.imag, z[..., 2 * n:]], -1)
        pair = torch.view_as_complex(z[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * by
        return torch.cat([torch.view_as_real(pair).flatten(-2), z[..., 2 * n:]], -1)

    out, dqkv = {}, []
    for i, (name, w) in enumerate((("q", st["wq"]), ("k", st["wk"]))):
        x, w = (t.double().requires_grad_(train) for t in (st["parts"][i], w))
        y = forward(x, w)
        out[name] = y.detach()
        if train:
            dx, out["dw" + name] = torch.autograd.grad(y, (x, w), st["grads"][i].double())
            dqkv.append(dx.flatten(2))
        del x, y
    out["v"] = st["parts"][2].double()
    if train:
        out["dqkv"] = torch.cat([*dqkv, st["grads"][2].double().flatten(2)], -1)
    return out


def _exact_dense(case, st):
    if 2 * case["M"] * case["K"] * case["N"] * (1 + case["gate"]) * 3 > 1.2e13:
        return None
    f = torch.nn.functional
    act = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
           "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}[case["act"]]
    train = case["dir"] == "train"
    names = [n for n in ("x", "w", "w_gate", "bias", "bias_gate", "residual") if st[n] is not None]
    t = {n: st[n].double().requires_grad_(train and n != "residual") for n in names}

    def product(w, b):
        z = torch.matmul(t["x"], t[w])
        return z + t[b] if b in t else z

    y = act(product("w", "bias"))
    if "w_gate" in t:
        y = y * product("w_gate", "bias_gate")
    if "residual" in t:
        y = y + t["residual"]
    out = dict(y=y.detach())
    if train:
        wanted = [n for n in names if n != "residual"]
        short = dict(x="dx", w="dw", w_gate="dw_gate", bias="db", bias_gate="db_gate")
        for n, g in zip(wanted, torch.autograd.grad(y, [t[n] for n in wanted], st["dy"].double())):
            out[short[n]] = g
    return out


def _exact_clip(case, st):
    squares = [torch.dot(t.double().flatten(), t.double().flatten()) for t in st["grads"]]
    norm = torch.sqrt(torch.stack(squares).sum())
    by = min(1.0, st["max_norm"] / (float(norm) + 1e-6))
    return dict({f"g{i}": t.double() * by for i, t in enumerate(st["grads"])}, norm=norm)
