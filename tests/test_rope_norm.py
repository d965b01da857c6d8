"""Norms of heads with the rotary turn behind them against the definition in 64 bits.

Tolerances.  The sum of D squares is off by at most (D / 2 + 8) 2^-24 of itself (it is formed by lanes),
rstd by half that and two units, so x^ = x rstd by e = (D / 2 + 16) 2^-24 of itself; the turn adds
2^-19 of a pair's norm (test_rope.py).  Rounding to the output's type adds eps / 2 of the value.

Backward, dz carries 2^-19 of the pair's norm, mean(w dz x^) the same and D 2^-24 of the mean of the
magnitudes: dx is off by (2^-18 + (2 D + 64) 2^-24) rstd (|w dz| + |x^| mean |w dz x^|), |dz| taken as
its pair's norm.  dw is a sum of rows by threads, then by the groups of a CTA, then by CTAs: at the
sizes below at most 1000 additions one behind the other, each 2^-24 of the sum of magnitudes."""
import math

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build
from deterministic_attention_backward_gb300.rope import _PART, _two

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
gpu = pytest.mark.gpu
EPS = 1e-5


def turned(z, f, m, pos, layout, back=False):
    """z [B,S,H,D] float64 turned, and each element's pair norm times m."""
    n = f.numel()
    a = pos.double()[:, :, None, None] * f
    c, s = a.cos() * m, a.sin() * (-m if back else m)
    i = torch.arange(n, device=z.device)
    lo, hi = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    out, norm = z.clone(), z.abs()
    out[..., lo] = z[..., lo] * c - z[..., hi] * s
    out[..., hi] = z[..., hi] * c + z[..., lo] * s
    r = (z[..., lo] ** 2 + z[..., hi] ** 2).sqrt() * m
    norm[..., lo] = r
    norm[..., hi] = r
    return out, norm


def xhat(x, eps=EPS):
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return x * rstd, rstd


def forward(x, w, f, m, pos, layout, eps=EPS):
    return turned(xhat(x, eps)[0] * w, f, m, pos, layout)


def inside(got, ref, tol, name=""):
    if got.dtype != F32:
        fi = torch.finfo(got.dtype)
        tol = tol + fi.eps / 2 * (ref.abs() + tol) + fi.smallest_normal * fi.eps
    else:
        tol = tol + 2.0 ** -24 * ref.abs()
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (name, (err - tol).max().item(), err.max().item())


def check_forward(y, x, w, f, m, pos, layout):
    D = x.shape[-1]
    ref, norm = forward(x.double(), w.double(), f, m, pos, layout)
    inside(y, ref, (2.0 ** -19 + (D / 2 + 16) * 2.0 ** -24) * norm)


def check_backward(dx, dw, dy, x, w, f, m, pos, layout):
    D = x.shape[-1]
    X, W = x.double(), w.double()
    dz, size = turned(dy.double(), f, m, pos, layout, back=True)
    h, rstd = xhat(X)
    ref = rstd * (W * dz - h * (W * dz * h).mean(-1, keepdim=True))
    tol = rstd * ((W * size).abs() + h.abs() * (W * size * h).abs().mean(-1, keepdim=True))
    inside(dx, ref, (2.0 ** -18 + (2 * D + 64) * 2.0 ** -24) * tol, "dx")
    if dw is not None:
        inside(dw, (dz * h).sum((0, 1, 2)),
               (2.0 ** -18 + (D + 1000) * 2.0 ** -24) * (size * h).abs().sum((0, 1, 2)), "dw")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def make(shape, dtype, seed, by=1.0, plus=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * by + plus).to(dtype)


def test_reference_gradient():
    """The gradient's formula above against central differences."""
    g = torch.Generator().manual_seed(0)
    x, dy = (torch.randn(1, 3, 2, 10, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(10, generator=g, dtype=torch.float64)
    f, pos = torch.tensor([1.0, 0.3, 0.01], dtype=torch.float64), torch.tensor([[5, 9, -2]])
    for layout in ("half", "interleaved"):
        dz, _ = turned(dy, f, 1.3, pos, layout, back=True)
        h, rstd = xhat(x)
        dx = rstd * (w * dz - h * (w * dz * h).mean(-1, keepdim=True))
        dw = (dz * h).sum((0, 1, 2))
        for t, d in ((x, dx), (w, dw)):
            u = torch.randn(t.shape, generator=g, dtype=torch.float64)

            def along(e):
                a, b = (x + e * u, w) if t is x else (x, w + e * u)
                return (forward(a, b, f, 1.3, pos, layout)[0] * dy).sum()
            slope = (along(1e-6) - along(-1e-6)) / 2e-6
            assert abs(slope - (d * u).sum()) < 1e-7


def test_abi_refusals(L):
    at = 1 << 20  # never dereferenced: every call below is refused first

    def part(inp=at, out=2 * at, heads=2, D=16, turn=1, stride=16):
        return _PART.pack(inp, out, heads, D, turn, *[stride] * 6)

    def fwd(parts=None, n=1, w=(0, 0), B=1, S=1, rot=8, layout=0, dtype=0, wdtype=0, freq=8 * at,
            pos=None, pos64=0):
        ws = _two(None, None)
        ws[0], ws[1] = w
        return L.dash_rope_norm_fwd(parts or part(), n, ws, B, S, rot, layout, dtype, wdtype, freq,
                                    1.0, 1e-5, pos, pos64, 0, 1, 0, None)
    for bad in (dict(n=0), dict(n=4), dict(B=0), dict(S=-1), dict(rot=7), dict(rot=0), dict(rot=18),
                dict(layout=2), dict(dtype=3), dict(wdtype=1), dict(freq=0), dict(freq=at + 4),
                dict(pos=at + 2), dict(pos=at + 4, pos64=1), dict(w=(at + 1, 0)),
                dict(parts=part(inp=0)), dict(parts=part(out=0)), dict(parts=part(inp=at + 1)),
                dict(parts=part(heads=0)), dict(parts=part(D=0)), dict(parts=part(turn=0)),
                dict(parts=part(out=at + 32)), dict(parts=part(out=8 * at)),
                dict(parts=part() + part(out=4 * at) + part(out=6 * at), n=3),
                dict(parts=part() * 2, n=2), dict(w=(2 * at, 0)),
                # the second part's weight in its output, the first being copied
                dict(parts=part(turn=0) + part(inp=4 * at, out=5 * at), n=2, w=(5 * at, 0))):
        assert fwd(**bad) == 1, bad
    assert fwd(parts=part(D=514)) == 2 and fwd(B=1 << 20, S=1 << 12) == 2

    def bwd(parts=None, x=None, n=1, w=(0, 0), dw=(0, 0), ws=64 * at, bytes=1 << 20, **k):
        wp, dp = _two(None, None), _two(None, None)
        wp[0], wp[1] = w
        dp[0], dp[1] = dw
        return L.dash_rope_norm_bwd(parts or part(), part(inp=3 * at) if x is None else x, n, wp, dp, 1,
                                    1, 8, 0, 0, 0, 8 * at, 1.0, 1e-5, None, 0, 0, 1, 0, ws, bytes, None)
    for bad in (dict(x=part(inp=0)), dict(x=part(inp=3 * at, D=18)), dict(x=part(inp=2 * at)),
                dict(dw=(5 * at + 1, 0)), dict(dw=(2 * at, 0)), dict(dw=(3 * at, 0)),
                dict(w=(5 * at, 0), dw=(5 * at, 0)), dict(dw=(64 * at, 0)), dict(ws=3 * at, dw=(at * 5, 0))):
        assert bwd(**bad) == 1, bad
    assert bwd(dw=(5 * at, 0), bytes=15) == 5 and bwd(dw=(5 * at, 0), ws=0) == 5
    two = part() + part(inp=4 * at, out=5 * at, D=24)
    assert bwd(parts=two, x=part(inp=6 * at) + part(inp=7 * at, D=24), n=2, dw=(9 * at, 10 * at)) == 2
    assert L.dash_rope_norm_bwd_workspace_bytes(0) == 0
    assert L.dash_rope_norm_bwd_workspace_bytes(513) == 0


CASES = [  # B, S, H, Hkv, D, rot, layout
    (1, 1, 1, 1, 2, 2, "half"),
    (1, 1, 32, 8, 128, 128, "half"),
    (2, 3, 4, 2, 64, 64, "interleaved"),
    (1, 5, 3, 1, 96, 48, "interleaved"),
    (2, 7, 2, 2, 20, 10, "half"),            # single elements
    (2, 7, 5, 1, 50, 24, "interleaved"),
    (1, 9, 2, 1, 127, 126, "half"),
    (1, 33, 5, 5, 128, 32, "half"),
    (2, 40, 3, 1, 24, 16, "half"),
    (1, 11, 2, 2, 512, 512, "half"),
    (1, 6, 2, 1, 510, 100, "interleaved"),
    (3, 1237, 4, 2, 64, 32, "interleaved"),
    (1, 2500, 3, 1, 256, 256, "half"),
    (2, 4096, 16, 4, 128, 128, "half"),
]


@gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_matches_definition(L, case, dtype):
    B, S, H, Hkv, D, rot, layout = case
    f, m = dash.rope_freqs(rot, scaling="ramp", factor=4.0)
    q, k, v = (make((B, S, h, D), dtype, i, 1.5) for i, h in enumerate((H, Hkv, Hkv)))
    dq, dk, dv = (make((B, S, h, D), dtype, i + 5) for i, h in enumerate((H, Hkv, Hkv)))
    wtype = F32 if S % 2 else dtype
    wq, wk = (make((D,), wtype, i + 9, 0.2, 1.0) for i in range(2))
    pos = torch.arange(S, device="cuda").expand(B, S) + 1000003
    a = dict(q_weight=wq, k_weight=wk, inv_freq=f, magnitude=m, start=1000003, layout=layout)
    y = dash.rope_norm_fwd(q, k, v, **a)
    for got, x, w in zip(y, (q, k), (wq, wk)):
        check_forward(got, x, w, f, m, pos, layout)
    assert torch.equal(y[2], v) and y[2].data_ptr() != v.data_ptr()
    assert all(t.is_contiguous() for t in y)
    g = dash.rope_norm_bwd(dq, dk, dv, q, k, **a)
    check_backward(g[0], g[3], dq, q, wq, f, m, pos, layout)
    check_backward(g[1], g[4], dk, k, wk, f, m, pos, layout)
    assert torch.equal(g[2], dv) and g[3].dtype == wtype
    again = dash.rope_norm_bwd(dq, dk, dv, q, k, **a)
    assert all(torch.equal(s, t) for s, t in zip(g, again))


@gpu
def test_parts_weights_and_positions(L):
    """q alone, one weight, none; given positions in any order, per batch and shared, strided; packed
    heads; a v of another size."""
    f, _ = dash.rope_freqs(32)
    q, k, dq = make((2, 6, 3, 64), F32, 0), make((2, 6, 1, 64), F32, 1), make((2, 6, 3, 64), F32, 2)
    w, one = make((64,), F32, 3, 0.2, 1.0), torch.ones(64, device="cuda")
    pos = torch.tensor([[5, 5, 0, -7, 2 ** 31 - 1, 123456789], [0, 1, 2, 3, 4, -2 ** 31]],
                       device="cuda")
    y = dash.rope_norm_fwd(q, q_weight=w, inv_freq=f, positions=pos)
    assert y[1] is None and y[2] is None
    check_forward(y[0], q, w, f, 1.0, pos, "half")
    y32 = dash.rope_norm_fwd(q, q_weight=w, inv_freq=f, positions=pos.int())
    assert torch.equal(y32[0], y[0])
    wide = torch.zeros(2, 12, dtype=torch.int64, device="cuda")
    wide[:, ::2] = pos
    assert torch.equal(dash.rope_norm_fwd(q, q_weight=w, inv_freq=f, positions=wide[:, ::2])[0], y[0])
    check_forward(dash.rope_norm_fwd(q, inv_freq=f, positions=pos[0])[0], q, one, f, 1.0,
                  pos[:1].expand(2, 6), "half")
    packed = dash.rope_norm_fwd(q.view(12, 3, 64), q_weight=w, inv_freq=f, positions=pos.reshape(12))[0]
    assert torch.equal(packed.view(2, 6, 3, 64), y[0])
    v = make((2, 6, 2, 40), F32, 4)
    q2, k2, v2 = dash.rope_norm_fwd(q, k, v, k_weight=w, inv_freq=f, positions=pos)
    check_forward(q2, q, one, f, 1.0, pos, "half")
    check_forward(k2, k, w, f, 1.0, pos, "half")
    assert torch.equal(v2, v)
    g = dash.rope_norm_bwd(dq, make((2, 6, 1, 64), F32, 5), v, q, k, k_weight=w, inv_freq=f,
                           positions=pos)
    assert g[3] is None and torch.equal(g[2], v)
    check_backward(g[0], None, dq, q, one, f, 1.0, pos, "half")
    check_backward(g[1], g[4], make((2, 6, 1, 64), F32, 5), k, w, f, 1.0, pos, "half")
    g = dash.rope_norm_bwd(dq, None, None, q, q_weight=w, inv_freq=f, positions=pos)
    check_backward(g[0], g[3], dq, q, w, f, 1.0, pos, "half")


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("offset", [0, 1])
def test_strided_views_and_in_place(L, dtype, offset):
    """Views of one qkv product in, views of its gradient out (whose surroundings stay), gradients
    written over the ones they come from."""
    B, S, H, Hkv, D = 2, 37, 4, 2, 64
    f, _ = dash.rope_freqs(D)
    width = (H + 2 * Hkv) * D

    def views(t):
        return tuple(p.unflatten(-1, (-1, D)) for p in
                     t[..., offset: offset + width].split([H * D, Hkv * D, Hkv * D], dim=-1))
    qkv, dqkv = (make((B, S, width + 8), dtype, i) for i in (3, 4))
    parts, grads = views(qkv), views(dqkv)
    w = make((D,), dtype, 5, 0.2, 1.0)
    a = dict(q_weight=w, k_weight=w, inv_freq=f, start=11)
    want = dash.rope_norm_fwd(*[t.contiguous() for t in parts], **a)
    gwant = dash.rope_norm_bwd(*[t.contiguous() for t in grads], *[t.contiguous() for t in parts[:2]],
                               **a)

    def same(s, t):
        if offset and dtype == F32:  # lanes hold other elements: sums in another order
            return torch.allclose(s, t, rtol=2 ** -16, atol=2 ** -18)
        return torch.equal(s, t) if not offset else \
            torch.allclose(s.float(), t.float(), rtol=2 ** -7, atol=2 ** -8)
    assert all(map(same, want, dash.rope_norm_fwd(*parts, **a)))
    for fn, args, ref in ((dash.rope_norm_fwd, parts, want),
                          (dash.rope_norm_bwd, (*grads, *parts[:2]), gwant)):
        out = torch.full_like(qkv, 7.0)
        res = fn(*args, out=views(out), **a)
        assert all(r.data_ptr() == t.data_ptr() for r, t in zip(res, views(out)))
        assert all(map(same, ref, res))
        assert (out[..., :offset] == 7).all() and (out[..., offset + width:] == 7).all()
    mine = tuple(t.clone() for t in want)
    src = tuple(t.contiguous() for t in parts)
    for t, s in zip(mine, src):
        t.copy_(s)
    res = dash.rope_norm_fwd(*mine, out=mine, **a)
    assert all(torch.equal(s, t) for s, t in zip(res, want))
    g = tuple(t.contiguous().clone() for t in grads)
    res = dash.rope_norm_bwd(*g, *src[:2], out=g, **a)
    assert all(torch.equal(s, t) for s, t in zip(res, gwant))


@gpu
def test_nothing_to_do_and_special_values(L):
    f, _ = dash.rope_freqs(64)
    w = torch.ones(64, dtype=BF, device="cuda")
    for shape in ((0, 4, 2, 64), (2, 0, 2, 64), (2, 4, 0, 64)):
        e = torch.zeros(shape, dtype=BF, device="cuda")
        k = torch.zeros(*shape[:2], 1, 64, dtype=BF, device="cuda")
        y = dash.rope_norm_fwd(e, k, k, q_weight=w, k_weight=w, inv_freq=f)
        assert y[0].shape == shape and y[1].shape == k.shape
        g = dash.rope_norm_bwd(e, k, k, e, k, q_weight=w, k_weight=w, inv_freq=f)
        assert g[0].shape == shape and (g[3] == 0).all() and (g[4] == 0).all()
    x = make((1, 4, 2, 64), BF, 0)
    x[0, 1, 0, 3] = math.nan
    x[0, 2, 1] = 0.0
    y = dash.rope_norm_fwd(x, q_weight=w, inv_freq=f, start=1)[0]
    bad = torch.zeros(1, 4, 2, dtype=torch.bool, device="cuda")
    bad[0, 1, 0] = True
    assert torch.equal(~y.isfinite().all(-1), bad) and (y[0, 2, 1] == 0).all()
    f2 = f.clone()
    f2[5] = math.inf
    y = dash.rope_norm_fwd(make((1, 4, 2, 64), BF, 0), q_weight=w, inv_freq=f2, start=1)[0]
    assert y.isnan().sum() == 4 * 2 * 2 and y[..., [5, 37]].isnan().all()


@gpu
def test_streams_and_graphs(L):
    f, _ = dash.rope_freqs(128)
    q, k, v = (make((1, 300, h, 128), BF, i) for i, h in enumerate((8, 2, 2)))
    w = make((128,), BF, 5, 0.2, 1.0)
    a = dict(q_weight=w, k_weight=w, inv_freq=f)
    want = dash.rope_norm_fwd(q, k, v, **a)
    gwant = dash.rope_norm_bwd(*want, q, k, **a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = dash.rope_norm_fwd(q, k, v, stream=s, **a)
    g = dash.rope_norm_bwd(*y, q, k, stream=s, **a)
    s.synchronize()
    assert all(torch.equal(p, r) for p, r in zip((*y, *g), (*want, *gwant)))
    ws = torch.empty(dash.rope_norm_bwd_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dash.rope_norm_fwd(q, k, v, **a)
        g = dash.rope_norm_bwd(*y, q, k, workspace=ws, **a)
    q.copy_(make((1, 300, 8, 128), BF, 20))
    ws.fill_(255)
    graph.replay()
    want = dash.rope_norm_fwd(q, k, v, **a)
    gwant = dash.rope_norm_bwd(*want, q, k, **a)
    assert all(torch.equal(p, r) for p, r in zip((*y, *g), (*want, *gwant)))


@gpu
def test_refusals(L):
    f, _ = dash.rope_freqs(32)
    q, k = make((2, 3, 2, 32), BF, 0), make((2, 3, 1, 32), BF, 1)
    w = torch.ones(32, dtype=BF, device="cuda")
    a = dict(q_weight=w, k_weight=w, inv_freq=f)
    for bad in (lambda: dash.rope_norm_fwd(q.cpu(), k, **a), lambda: dash.rope_norm_fwd(q, **a),
                lambda: dash.rope_norm_fwd(q, k, q_weight=w[:31], inv_freq=f),
                lambda: dash.rope_norm_fwd(q, k, q_weight=w.half(), inv_freq=f),
                lambda: dash.rope_norm_fwd(q, k, q_weight=w, k_weight=w.float(), inv_freq=f),
                lambda: dash.rope_norm_fwd(q[..., ::2], inv_freq=f),
                lambda: dash.rope_norm_fwd(q, inv_freq=f, layout="other"),
                lambda: dash.rope_norm_fwd(q, inv_freq=f, start=2 ** 63),
                lambda: dash.rope_norm_fwd(make((1, 1, 1, 520), BF, 0), inv_freq=f),
                lambda: dash.rope_norm_bwd(q, k, None, q, **a),
                lambda: dash.rope_norm_bwd(q, k, None, q[:1], k, **a),
                lambda: dash.rope_norm_bwd(q, k, None, q, k.float(), **a),
                lambda: dash.rope_norm_bwd(q, k, None, q, k, workspace=torch.empty(8, device="cuda"), **a),
                lambda: dash.rope_norm_bwd(q, k, None, q, k, out=(q[:1], None, None), **a)):
        with pytest.raises(ValueError):
            bad()
    y = torch.empty_like(q)
    with pytest.raises(dash.DashError):  # over the forward's input
        dash.rope_norm_bwd(y, None, None, q, out=(q, None, None), inv_freq=f)


@gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("case", [(2, 37, 4, 2, 64, 64, "half"), (1, 513, 4, 1, 128, 128, "interleaved"),
                                  (1, 300, 8, 8, 128, 32, "half"), (1, 3, 3, 1, 512, 512, "half"),
                                  (3, 70, 5, 1, 96, 48, "interleaved"), (1, 900, 2, 2, 256, 64, "half"),
                                  (2, 40, 3, 1, 24, 16, "half"), (1, 50, 3, 1, 50, 24, "half")], ids=str)
def test_bits_do_not_depend_on_the_place_in_memory(L, case, dtype):
    """The same heads at other places and strides give the same bits, their weights' gradients too; what
    lies beside them stays."""
    B, S, H, Hkv, D, rot, layout = case
    f, _ = dash.rope_freqs(rot)
    widths = [H * D, Hkv * D, Hkv * D]
    wq, wk = (make((D,), dtype, i, 0.2, 1.0) for i in (5, 6))
    a = dict(q_weight=wq, k_weight=wk, inv_freq=f, start=11, layout=layout)

    def parts(t, at):
        return tuple(p.unflatten(-1, (-1, D)) for p in
                     t[..., at:at + sum(widths)].split(widths, dim=-1))
    x, g = (make((B, S, sum(widths)), dtype, i) for i in (3, 4))
    want = dash.rope_norm_fwd(*parts(x, 0), **a)
    gwant = dash.rope_norm_bwd(*parts(g, 0), *parts(x, 0)[:2], **a)
    for at, room in ((1, 8), (2, 9), (4, 16), (8, 16), (0, 1)):
        def wide(t):
            big = torch.full((B, S, sum(widths) + room), 7.0, dtype=dtype, device="cuda")
            big[..., at:at + sum(widths)] = t
            return big
        for fn, args, ref in ((dash.rope_norm_fwd, parts(wide(x), at), want),
                              (dash.rope_norm_bwd, (*parts(wide(g), at), *parts(wide(x), at)[:2]), gwant)):
            out = wide(torch.zeros_like(x))
            assert all(map(torch.equal, fn(*args, **a), ref)), (fn.__name__, at, room)
            res = fn(*args, out=parts(out, at), **a)
            assert all(map(torch.equal, res, ref)), (fn.__name__, at, room)
            assert (out[..., :at] == 7).all() and (out[..., at + sum(widths):] == 7).all()
            # over the tensors themselves
            res = fn(*args, out=args[:3], **a)
            assert all(map(torch.equal, res, ref)), (fn.__name__, at, room)


@gpu
@pytest.mark.parametrize("which", ["q", "k"])
def test_workspace_is_of_the_heads_that_have_a_weight(L, which):
    """Heads of q and k of different sizes, a weight for one of them: its size decides."""
    f, _ = dash.rope_freqs(32)
    small, large = make((1, 64, 1, 32), BF, 0), make((1, 64, 8, 512), BF, 1)
    q, k = (large, small) if which == "q" else (small, large)
    dq, dk = make(q.shape, BF, 2), make(k.shape, BF, 3)
    w = make((512,), BF, 4, 0.2, 1.0)
    a = dict(inv_freq=f, **{which + "_weight": w})
    pos = torch.arange(64, device="cuda")[None]
    g = dash.rope_norm_bwd(dq, dk, None, q, k, **a)
    one = torch.ones(32, device="cuda")
    check_backward(g[0], g[3], dq, q, w if which == "q" else one, f, 1.0, pos, "half")
    check_backward(g[1], g[4], dk, k, w if which == "k" else one, f, 1.0, pos, "half")
    need = dash.rope_norm_bwd_workspace_bytes(512)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    again = dash.rope_norm_bwd(dq, dk, None, q, k, workspace=ws[:need], **a)
    assert all(p is r or torch.equal(p, r) for p, r in zip(g, again)) and (ws[need:] == 255).all()
    with pytest.raises(ValueError, match="workspace"):
        dash.rope_norm_bwd(dq, dk, None, q, k, workspace=ws[:need - 1], **a)


def test_abi_outputs_apart_from_everything_that_is_read(L):
    """The weights' gradients and the workspace are written while frequencies, positions and both weights
    are read: they lie apart from all of each, whichever part has a weight."""
    at = 1 << 20  # never dereferenced: every call below is refused

    def part(inp, out, D):
        return _PART.pack(inp, out, 2, D, 1, *[4096] * 6)

    def bwd(w=(0, 10 * at), dw=(0, 11 * at), ws=64 * at, bytes=1 << 20, pos=None):
        wp, dp = _two(None, None), _two(None, None)
        wp[0], wp[1] = w
        dp[0], dp[1] = dw
        return L.dash_rope_norm_bwd(part(at, 2 * at, 512) + part(3 * at, 4 * at, 16),
                                    part(5 * at, 5 * at, 512) + part(6 * at, 6 * at, 16), 2, wp, dp, 1, 4,
                                    8, 0, 0, 0, 8 * at, 1.0, 1e-5, pos, 1, 0, 1, 0, ws, bytes, None)
    assert bwd(bytes=15) == 5  # (as far as the workspace's size nothing is amiss)
    for bad in (dict(dw=(0, 8 * at + 16)), dict(ws=8 * at), dict(ws=9 * at, pos=9 * at),
                dict(dw=(0, 9 * at + 8), pos=9 * at), dict(ws=10 * at - 16),
                # the first part's weight, of 512 elements, behind what the second's gradient has
                dict(w=(12 * at, 10 * at), dw=(0, 12 * at + 512)),
                dict(w=(12 * at, 10 * at), ws=12 * at + 512)):
        assert bwd(**bad) == 1, bad
