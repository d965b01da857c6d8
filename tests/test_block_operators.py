"""The operators around the attention run together: through the synthetic block's options, forward
and every gradient against the same block in 64 bits, and called one after another as a layer
does, eagerly, on another stream and from captured graphs."""
import pytest
import torch
import torch.nn.functional as F

from deterministic_attention_backward_gb300 import block

gpu = pytest.mark.gpu

# The block rounds to bf16 at most 14 times from its input to its output (norms, the qkv product,
# rotary, probabilities, attention, head norm, five products, silu, gate, two joins) and as often
# again on the way back.  A rounding is off by half a step at most, 2^-8 of the value, spread evenly:
# 2^-8 / sqrt(3) in the root mean square.  Their sum, as if every one pointed the same way:
ROUND = 2.0 ** -8 / 3 ** 0.5
TOL_OUT, TOL_GRAD = 14 * ROUND, 28 * ROUND


def norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w


def turn(x, base):
    S, d = x.shape[1], x.shape[-1]
    f = base ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    a = torch.arange(S, device=x.device, dtype=torch.float64)[:, None, None] * f
    u, w = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()], -1)


def probs(q, k, causal):
    """[B, H, S, S] of q [B, S, H, d] and k [B, S, Hkv, d]."""
    k = k.repeat_interleave(q.shape[2] // k.shape[2], 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) * q.shape[-1] ** -0.5
    if causal:
        S = q.shape[1]
        s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1),
                          float("-inf"))
    return s.softmax(-1)


def plain(x, p, heads, kv_heads, D, rotary, causal):
    """The block in the type of its tensors."""
    B, S, _ = x.shape
    qkv = norm(x, p["n1"]) @ p["wqkv"]
    q, k, v = (t.unflatten(-1, (-1, D)) for t in
               qkv.split([heads * D, kv_heads * D, kv_heads * D], -1))
    def halves(t):
        return t.unflatten(-1, (2, D // 2)).unbind(-2)

    def mapped(q, k):
        return probs(turn(q, rotary), turn(k, rotary), causal) if rotary else probs(q, k, causal)
    if "lam" in p:
        (q1, q2), (k1, k2) = halves(q), halves(k)
        P = mapped(q1, k1) - p["lam"][:, None, None] * mapped(q2, k2)
    else:
        P = mapped(q, k)
    o = torch.einsum("bhij,bjhd->bihd", P, v.repeat_interleave(heads // kv_heads, 2))
    if "nh" in p:
        o = norm(o, p["nh"])
    a = o.reshape(B, S, heads * D) @ p["wo"]
    y = x + (norm(a, p["p1"]) if "p1" in p else a)
    hid = norm(y, p["n2"])
    m = (F.silu(hid @ p["w1"]) * (hid @ p["w3"])) @ p["w2"]
    return y + (norm(m, p["p2"]) if "p2" in p else m)


NAMES = ("wqkv", "wo", "w1", "w3", "w2", "n1", "n2", "p1", "p2", "lam", "nh")
OPTIONS = [
    dict(rotary=10000.0),
    dict(fused_norms=True),
    dict(fused_norms=True, post_norms=True),
    dict(differential=0.5),
    dict(rotary=10000.0, fused_norms=True, post_norms=True, differential=0.8),
]


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


@gpu
@pytest.mark.parametrize("options", OPTIONS, ids=lambda o: "+".join(o))
@pytest.mark.parametrize("D,S,causal", [(128, 200, True), (64, 129, False), (128, 1, True)])
def test_block_options(options, D, S, causal):
    if D == 64 and "differential" not in options:
        D = 128
    heads, kv_heads, hidden = 4, 2, 512
    blk = block.Block(hidden=hidden, heads=heads, kv_heads=kv_heads, head_dim=D, ffn=768, seed=3,
                      **options)
    g = torch.Generator().manual_seed(7)
    p = {n: getattr(blk, n) for n in NAMES if getattr(blk, n, None) is not None}
    with torch.no_grad():
        for n in ("n1", "n2", "p1", "p2", "lam", "nh"):
            if n in p:
                p[n].mul_((1 + 0.3 * torch.randn(p[n].shape, generator=g)).to(p[n]))
    x = torch.randn(2, S, hidden, generator=g).to("cuda", torch.bfloat16).requires_grad_()
    gout = torch.randn(2, S, hidden, generator=g).to("cuda", torch.bfloat16)
    out = blk(x, "shift_fill", causal)
    out.backward(gout)

    pd = {n: t.detach().double().requires_grad_() for n, t in p.items()}
    xd = x.detach().double().requires_grad_()

    def ref(xx, pp):
        return plain(xx, pp, heads, kv_heads, D, options.get("rotary"), causal)
    want = ref(xd, pd)
    want.backward(gout.double())
    # the reference's gradients against differences of itself
    with torch.no_grad():
        dirs = {n: torch.randn(t.shape, generator=g, dtype=torch.float64).cuda()
                for n, t in pd.items()}
        dx = torch.randn(xd.shape, generator=g, dtype=torch.float64).cuda()
        e = 1e-5

        def along(s):
            return (ref(xd + s * e * dx, {n: t + s * e * dirs[n] * t.abs().mean()
                                          for n, t in pd.items()}) * gout.double()).sum()
        slope = (along(1) - along(-1)) / (2 * e)
        terms = [(xd.grad * dx).sum()] + [(pd[n].grad * dirs[n]).sum() * pd[n].abs().mean()
                                          for n in pd]
        assert abs(slope - sum(terms)) <= 1e-5 * sum(t.abs() for t in terms)

    assert rel(out, want) <= TOL_OUT
    # with one token a head's output is (1 - lam) v, and its norm does not see lam
    errors = {n: rel(t.grad, pd[n].grad) for n, t in p.items() if n != "lam" or S > 1}
    errors["x"] = rel(x.grad, xd.grad)
    assert all(v <= TOL_GRAD for v in errors.values()), errors

    # again, with the same bits
    first = [t.grad for t in (x, *p.values())]
    for t in (x, *p.values()):
        t.grad = None
    blk(x, "shift_fill", causal).backward(gout)
    assert all(torch.equal(t.grad, g) for t, g in zip((x, *p.values()), first))


@gpu
def test_block_takes_expanded_gradients():
    """``sum().backward()`` hands in a gradient of strides 0."""
    got = []
    for whole in (False, True):
        blk = block.Block(hidden=512, heads=4, kv_heads=2, head_dim=128, ffn=768, rotary=100.0,
                          fused_norms=True, post_norms=True, differential=0.8)
        x = torch.linspace(-1, 1, 96 * 512, device="cuda").to(torch.bfloat16).view(1, 96, 512)
        x.requires_grad_()
        out = blk(x, "auto")
        out.backward(torch.ones_like(out)) if whole else out.sum().backward()
        got.append([x.grad] + [t.grad for t in blk.parameters()])
    for a, b in zip(*got):
        assert torch.equal(a, b)


class Layer:
    """The operators of one layer and their gradients, as a program without autograd calls them:
    a qkv product's output through rotary, differential attention, norm of heads and the join."""

    B, S, H, HKV, D = 2, 333, 4, 2, 128

    def __init__(self, dash, seed):
        self.dash = dash
        g = torch.Generator().manual_seed(seed)
        hidden, wide = self.H * self.D, (self.H + 2 * self.HKV) * self.D

        def rand(*shape, dtype=torch.bfloat16):
            return torch.randn(*shape, generator=g).to("cuda", dtype)
        self.qkv, self.x = rand(self.B, self.S, wide), rand(self.B, self.S, hidden)
        self.dy, self.dh = rand(self.B, self.S, hidden), rand(self.B, self.S, hidden)
        self.lam = torch.rand(self.H, generator=g).cuda()
        self.w_head, self.w_post, self.w_next = rand(self.D), rand(hidden), rand(hidden)
        self.freqs, self.magnitude = dash.rope_freqs(self.D // 2, scaling="ramp", factor=4.0)

    def inputs(self):
        return self.qkv, self.x, self.dy, self.dh

    def views(self, t):
        d = self.D // 2
        parts = t.split([self.H * self.D, self.HKV * self.D, self.HKV * self.D], -1)
        return [u.unflatten(-1, (-1, n)) for u, n in zip(parts, (d, d, self.D))]

    def __call__(self, **kw):
        dash, rot = self.dash, dict(inv_freq=self.freqs, magnitude=self.magnitude, **kw)
        q, k, v = dash.rope_fwd(*self.views(self.qkv), **rot)
        o, o2, lse = dash.diff_fwd(q, k, v, self.lam, causal=True, **kw)
        n, rstd = dash.norm_fwd(o, self.w_head, **kw)
        a = n.view(self.B, self.S, -1)
        w = dict(w_post=self.w_post, w_next=self.w_next, **kw)
        y, h, ra, ry = dash.join_fwd(self.x, a, **w)
        dx, da, dw_post, _, dw_next = dash.join_bwd(self.dy, self.dh, y, a, ra, ry, **w)
        do, dw_head = dash.norm_bwd(da.view_as(o), o, rstd, self.w_head, **kw)
        dq, dk, dv, dlam = dash.diff_bwd(q, k, v, o, o2, do, lse, self.lam, causal=True, **kw)
        dqkv = torch.empty_like(self.qkv)
        dash.rope_bwd(dq, dk, dv, out=self.views(dqkv), **rot)
        return y, h, dx, dqkv, dlam, dw_head, dw_post, dw_next

    def reference(self):
        leaves = [t.double().requires_grad_() for t in
                  (self.x, self.qkv, self.lam, self.w_head, self.w_post, self.w_next)]
        x, qkv, lam, w_head, w_post, w_next = leaves
        d = self.D // 2
        q, k, v = self.views(qkv)
        a = torch.arange(self.S, device="cuda", dtype=torch.float64)[:, None, None] * self.freqs

        def turned(t):
            u, w = t[..., :d // 2], t[..., d // 2:]
            return self.magnitude * torch.cat([u * a.cos() - w * a.sin(),
                                               w * a.cos() + u * a.sin()], -1)
        q, k = turned(q), turned(k)
        P = probs(q[:, :, 0::2], k[:, :, 0::2], True) - \
            lam[:, None, None] * probs(q[:, :, 1::2], k[:, :, 1::2], True)
        o = torch.einsum("bhij,bjhd->bihd", P, v.repeat_interleave(self.H // self.HKV, 2))
        br = norm(o, w_head).reshape(self.B, self.S, -1)
        y = x + norm(br, w_post)
        h = norm(y, w_next)
        grads = torch.autograd.grad([y, h], leaves, [self.dy.double(), self.dh.double()])
        return [t.detach() for t in (y, h)] + list(grads)


@gpu
def test_layer_against_formulas():
    import deterministic_attention_backward_gb300 as dash
    layer = Layer(dash, 11)
    names = ("y", "h", "dx", "dqkv", "dlam", "dw_head", "dw_post", "dw_next")
    # roundings on the way: 7 to h (rotary, P, o, norm, y, h and a join's branch), 7 back
    for name, got, ref in zip(names, layer(), layer.reference()):
        assert rel(got, ref) <= 14 * ROUND, name


@gpu
def test_layer_on_another_stream():
    import deterministic_attention_backward_gb300 as dash
    layer = Layer(dash, 12)
    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        here = layer()
    torch.cuda.synchronize()
    given = layer(stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, here, given):
        assert torch.equal(a, b) and torch.equal(a, c)


@gpu
def test_layers_in_captured_graphs():
    """Two layers captured, forward and backward, then replayed on new inputs, at once on two
    streams: each gives the eager call's bits."""
    import deterministic_attention_backward_gb300 as dash
    layers = [Layer(dash, 21), Layer(dash, 22)]
    streams = [torch.cuda.Stream() for _ in layers]
    for layer in layers:
        layer()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for layer in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer())
        graphs.append(graph)
    for layer in layers:
        for t in layer.inputs():
            t.mul_(0.75).add_(0.125)
    want = [layer() for layer in layers]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_block_refuses_options():
    with pytest.raises(ValueError, match="fused_norms"):
        block.Block(hidden=64, heads=1, kv_heads=1, head_dim=64, ffn=64, device="cpu",
                    post_norms=True)
    with pytest.raises(ValueError, match="heads of 64 or 128"):
        block.Block(hidden=64, heads=1, kv_heads=1, head_dim=32, ffn=64, device="cpu",
                    differential=0.8)


def test_block_options_leave_the_weights_alone():
    sizes = dict(hidden=128, heads=2, kv_heads=1, head_dim=64, ffn=128, device="cpu", seed=9)
    a = block.Block(**sizes)
    b = block.Block(**sizes, rotary=10000.0, fused_norms=True, post_norms=True, differential=0.8)
    assert len(a.parameters()) == 7 and len(b.parameters()) == 11
    for t, u in zip(a.parameters(), b.parameters()):
        assert torch.equal(t, u)
    assert b.freqs.shape == (16,) and torch.equal(b.lam, torch.full((2,), 0.8))
