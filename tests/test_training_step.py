"""A training step of the block with its heads' norms, products and clipping in this library's kernels:
through the block's options against the same block in 64 bits, and as a program without autograd calls
the operators one after another, eagerly, on another stream and from captured graphs."""
import pytest
import torch
import torch.nn.functional as F

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import block

gpu = pytest.mark.gpu

# As for the block with the other operators (test_block_operators.py): at most 14 roundings on the way,
# as many back, each 2^-8 / sqrt(3) of its value in the root mean square, all pointing the same way.
ROUND = 2.0 ** -8 / 3 ** 0.5
TOL_OUT, TOL_GRAD = 14 * ROUND, 28 * ROUND


def rel(got, ref):
    got, ref = got.detach(), ref.detach()
    return float((got.double() - ref).norm() / ref.norm())


def norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w


def turn(x, base):
    S, d = x.shape[1], x.shape[-1]
    f = base ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    a = torch.arange(S, device=x.device, dtype=torch.float64)[:, None, None] * f
    u, w = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()], -1)


def attention(q, k, v, causal=True):
    G = q.shape[2] // k.shape[2]
    k, v = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) * q.shape[-1] ** -0.5
    if causal:
        S = q.shape[1]
        s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    return torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v)


def plain(x, p, heads, kv_heads, D, rotary):
    """The block in the type of its tensors."""
    B, S, _ = x.shape
    qkv = norm(x, p["n1"]) @ p["wqkv"]
    q, k, v = (t.unflatten(-1, (-1, D)) for t in
               qkv.split([heads * D, kv_heads * D, kv_heads * D], -1))
    if "nq" in p:
        q, k = norm(q, p["nq"]), norm(k, p["nk"])
    if rotary:
        q, k = turn(q, rotary), turn(k, rotary)
    y = x + attention(q, k, v).reshape(B, S, heads * D) @ p["wo"]
    hid = norm(y, p["n2"])
    return y + (F.silu(hid @ p["w1"]) * (hid @ p["w3"])) @ p["w2"]


NAMES = ("wqkv", "wo", "w1", "w3", "w2", "n1", "n2", "nq", "nk")
OPTIONS = [
    dict(rotary=10000.0, qk_norm=True),
    dict(fused_dense=True),
    dict(fused_dense=True, fused_norms=True),
    dict(rotary=500.0, qk_norm=True, fused_dense=True),
    dict(rotary=10000.0, qk_norm=True, fused_dense=True, fused_norms=True),
]


@gpu
@pytest.mark.parametrize("options", OPTIONS, ids=lambda o: "+".join(o))
@pytest.mark.parametrize("S", [200, 129, 1])
def test_block_options(options, S):
    heads, kv_heads, hidden, D = 4, 2, 512, 128
    blk = block.Block(hidden=hidden, heads=heads, kv_heads=kv_heads, head_dim=D, ffn=776, seed=3,
                      **options)
    g = torch.Generator().manual_seed(7)
    p = {n: getattr(blk, n) for n in NAMES if getattr(blk, n, None) is not None}
    with torch.no_grad():
        for n in ("n1", "n2", "nq", "nk"):
            if n in p:
                p[n].mul_((1 + 0.3 * torch.randn(p[n].shape, generator=g)).to(p[n]))
    x = torch.randn(2, S, hidden, generator=g).to("cuda", torch.bfloat16).requires_grad_()
    gout = torch.randn(2, S, hidden, generator=g).to("cuda", torch.bfloat16)
    out = blk(x, "shift_fill")
    out.backward(gout)
    pd = {n: t.detach().double().requires_grad_() for n, t in p.items()}
    xd = x.detach().double().requires_grad_()
    want = plain(xd, pd, heads, kv_heads, D, options.get("rotary"))
    want.backward(gout.double())
    assert rel(out, want) <= TOL_OUT
    # of a single token only the value matters: q and k have no gradient to speak of
    errors = {n: rel(t.grad, pd[n].grad) for n, t in p.items()
              if S > 1 or n not in ("nq", "nk")}
    errors["x"] = rel(x.grad, xd.grad)
    assert all(v <= TOL_GRAD for v in errors.values()), errors
    grads = [t.grad for t in (x, *p.values())]
    for t in (x, *p.values()):
        t.grad = None
    blk(x, "shift_fill").backward(gout)
    assert all(torch.equal(t.grad, g) for t, g in zip((x, *p.values()), grads))
    # and the step's end: all of them clipped
    mine = [t.grad.clone() for t in blk.parameters()]
    total = float(torch.cat([t.double().flatten() for t in mine]).norm())
    got = blk.clip(0.5 * total)
    assert abs(float(got) - total) <= 2.0 ** -17 * total
    for t, g in zip(blk.parameters(), mine):
        ref = g.double() * 0.5
        assert ((t.grad.double() - ref).abs() <= (2.0 ** -9 + 2.0 ** -16) * ref.abs()).all()


@gpu
def test_block_takes_expanded_gradients():
    got = []
    for whole in (False, True):
        blk = block.Block(hidden=512, heads=4, kv_heads=2, head_dim=128, ffn=768, rotary=100.0,
                          qk_norm=True, fused_dense=True)
        x = torch.linspace(-1, 1, 96 * 512, device="cuda").to(torch.bfloat16).view(1, 96, 512)
        x.requires_grad_()
        out = blk(x, "auto")
        out.backward(torch.ones_like(out)) if whole else out.sum().backward()
        got.append([x.grad] + [t.grad for t in blk.parameters()])
    for a, b in zip(*got):
        assert torch.equal(a, b)


class Step:
    """A layer's forward, backward and clipping as a program without autograd calls them."""

    B, S, H, HKV, D, FFN = 2, 190, 4, 2, 64, 520

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        hidden, wide = self.H * self.D, (self.H + 2 * self.HKV) * self.D

        def rand(*shape, by=1.0, plus=0.0):
            return (torch.randn(*shape, generator=g) * by + plus).to("cuda", torch.bfloat16)
        self.x, self.dy = rand(self.B, self.S, hidden), rand(self.B, self.S, hidden)
        self.wqkv, self.wo = rand(hidden, wide, by=hidden ** -0.5), rand(hidden, hidden,
                                                                         by=hidden ** -0.5)
        self.w1, self.w3 = (rand(self.FFN, hidden, by=hidden ** -0.5).t() for _ in range(2))
        self.w2, self.b2 = rand(self.FFN, hidden, by=self.FFN ** -0.5), rand(hidden)
        self.nq, self.nk = rand(self.D, by=0.2, plus=1.0), rand(self.D, by=0.2, plus=1.0)
        self.freqs, _ = dash.rope_freqs(self.D)

    def inputs(self):
        return self.x, self.dy

    def views(self, t):
        parts = t.split([self.H * self.D, self.HKV * self.D, self.HKV * self.D], -1)
        return [u.unflatten(-1, (-1, self.D)) for u in parts]

    def __call__(self, **kw):
        rot = dict(q_weight=self.nq, k_weight=self.nk, inv_freq=self.freqs, **kw)
        qkv, _ = dash.dense_fwd(self.x, self.wqkv, **kw)
        q, k, v = dash.rope_norm_fwd(*self.views(qkv), **rot)
        o, lse = dash.fwd(q, k, v, causal=True, **kw)
        flat = o.view(self.B, self.S, -1)
        y, _ = dash.dense_fwd(flat, self.wo, residual=self.x, **kw)
        m, kept = dash.dense_fwd(y, self.w1, act="silu", w_gate=self.w3, **kw)
        z, _ = dash.dense_fwd(m, self.w2, self.b2, residual=y, **kw)
        dm, dw2, db2, _, _ = dash.dense_bwd(self.dy, m, self.w2, bias=self.b2, **kw)
        dy, dw1, _, dw3, _ = dash.dense_bwd(dm, y, self.w1, kept, act="silu", w_gate=self.w3, **kw)
        dy = self._add(dy, self.dy, kw)  # the residual stream's
        do, dwo, *_ = dash.dense_bwd(dy, flat, self.wo, **kw)
        dq, dk, dv = dash.bwd(q, k, v, o, do.view_as(o), lse, causal=True, schedule="auto", **kw)
        dqkv = torch.empty_like(qkv)
        *_, dnq, dnk = dash.rope_norm_bwd(dq, dk, dv, *self.views(qkv)[:2],
                                          out=self.views(dqkv), **rot)
        dx, dwqkv, *_ = dash.dense_bwd(dqkv, self.x, self.wqkv, **kw)
        dx = self._add(dx, dy, kw)
        grads = [dwqkv, dwo, dw1, dw3, dw2, db2, dnq, dnk]
        # below the norm that these have, so that they are clipped
        return (z, dx, dash.grad_clip(grads, 1.0, **kw), *grads)

    @staticmethod
    def _add(a, b, kw):
        with torch.cuda.stream(kw.get("stream")):
            return a + b

    def reference(self):
        leaves = [t.double().requires_grad_() for t in
                  (self.x, self.wqkv, self.wo, self.w1, self.w3, self.w2, self.b2, self.nq, self.nk)]
        x, wqkv, wo, w1, w3, w2, b2, nq, nk = leaves
        q, k, v = self.views(x @ wqkv)
        q, k = turn(norm(q, nq), 10000.0), turn(norm(k, nk), 10000.0)
        y = x + attention(q, k, v).reshape(self.B, self.S, -1) @ wo
        z = y + (F.silu(y @ w1) * (y @ w3)) @ w2 + b2
        grads = torch.autograd.grad(z, leaves, self.dy.double())
        dx, *grads = grads
        total = torch.cat([t.flatten() for t in grads]).norm()
        return [z.detach(), dx, total, *[t / (total + 1e-6) for t in grads]]


@gpu
def test_step_against_formulas():
    step = Step(11)
    got, ref = step(), step.reference()
    assert float(ref[2]) > 1.0
    names = ("z", "dx", "norm", "dwqkv", "dwo", "dw1", "dw3", "dw2", "db2", "dnq", "dnk")
    for i, name in enumerate(names):
        assert rel(got[i], ref[i]) <= (TOL_OUT if name in ("z", "norm") else TOL_GRAD), name


@gpu
def test_step_on_another_stream():
    step = Step(12)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        here = step()
    torch.cuda.synchronize()
    given = step(stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, here, given):
        assert torch.equal(a, b) and torch.equal(a, c)


@gpu
def test_steps_in_captured_graphs():
    """Two steps captured, then replayed on new inputs, at once on two streams: each gives the eager
    call's bits."""
    steps = [Step(21), Step(22)]
    streams = [torch.cuda.Stream() for _ in steps]
    for step in steps:
        step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for step in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for step in steps:
        for t in step.inputs():
            t.mul_(0.75).add_(0.125)
    want = [step() for step in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_block_options_on_the_host():
    sizes = dict(hidden=128, heads=2, kv_heads=1, head_dim=64, ffn=128, device="cpu", seed=9)
    a = block.Block(**sizes)
    b = block.Block(**sizes, rotary=10000.0, qk_norm=True, fused_dense=True)
    assert len(a.parameters()) == 7 and len(b.parameters()) == 9
    assert b.nq.shape == (64,) and (b.nk == 1).all()
    for t, u in zip(a.parameters(), b.parameters()):
        assert torch.equal(t, u)
    with pytest.raises(ValueError, match="rotary"):
        block.Block(**sizes, qk_norm=True)


def test_block_keeps_nothing_where_no_backward_follows(monkeypatch):
    """What the backward of a product needs is kept only where gradients are on and one of its operands has
    one."""
    asked = []

    def dense_fwd(x, w, *, act, w_gate, residual, keep=True):
        asked.append(keep)
        return torch.zeros(*x.shape[:-1], w.shape[1]), None
    monkeypatch.setattr(dash, "dense_fwd", dense_fwd, raising=False)
    blk = block.Block(hidden=128, heads=2, kv_heads=1, head_dim=64, ffn=128, device="cpu", fused_dense=True)
    x = torch.zeros(1, 3, 128)
    assert blk.Dense.call(x, blk.w1, blk.w3, act="silu").requires_grad and asked.pop()
    with torch.no_grad():
        assert not blk.Dense.call(x, blk.w1, blk.w3, act="silu").requires_grad and not asked.pop()
    assert not blk.Dense.call(x, blk.w1.detach(), blk.w3.detach()).requires_grad and not asked.pop()
    assert blk.Dense.call(x, blk.w1.detach(), residual=x[..., :128].clone().requires_grad_()).requires_grad
    assert asked.pop() and not asked


@gpu
def test_block_without_gradients_gives_the_same_bits():
    for options in (dict(fused_dense=True), dict(rotary=100.0, qk_norm=True, fused_dense=True, fused_norms=True)):
        blk = block.Block(hidden=512, heads=4, kv_heads=2, head_dim=128, ffn=776, **options)
        x = torch.linspace(-1, 1, 96 * 512, device="cuda").to(torch.bfloat16).view(1, 96, 512)
        with torch.no_grad():
            y = blk(x, "auto")
        assert not y.requires_grad and torch.equal(blk(x, "auto"), y)
