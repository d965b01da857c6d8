"""Products with their epilogue against the definition in 64 bits.

Tolerances.  Products of 16-bit values are exact in fp32.  The tensor core adds 16 of them to an
accumulator at a time; an addition that aligns its terms to the largest and cuts them off errs by less
than 2^-22 of the sum of their magnitudes, over K / 16 steps and the additions of splits and parts
behind them: (K / 16 + 40) 2^-22 S with S = sum |x| |w|.  The activations' slopes are below 1.13 and
their functions good to 2^-20 of |z| + 1.  A rounding to the type is off by eps / 2 of the value.  The
backward rounds dz (and dgate) once before its products, which enters as eps / 2 sum |dz| |w|.

That bound holds for every element, but roundings rarely all point one way: in the norm over a tensor a
rounding counts as its root mean square, eps / 2 / sqrt 3 of the values' norm, so dx and dw, with two
roundings one behind the other, are held to twice that, and the sums' own error, as well."""
import math

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build
from deterministic_attention_backward_gb300.dense import _BWD, _FWD

BF, HF = torch.bfloat16, torch.float16
gpu = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def act_of(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    t = torch.tanh(u)
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * math.sqrt(2 / math.pi) * (
        1 + 3 * 0.044715 * z * z)


def step(t):
    return torch.finfo(t).eps / 2


def rounded(ref, tol, dtype):
    return tol + step(dtype) * (ref.abs() + tol) + torch.finfo(dtype).smallest_normal * \
        torch.finfo(dtype).eps


def sums(K):
    return (K / 16 + 40) * 2.0 ** -22


def inside(got, ref, tol, name=""):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (name, (err - tol).max().item(), err.max().item())


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def make(shape, dtype, seed, by=1.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=device) * by).to(dtype)


def weight(K, N, order, dtype, seed):
    w = make((K, N), dtype, seed, K ** -0.5)
    return w if order == "kn" else w.t().contiguous().t()


def unpacked(kept, rows, N):
    """What the forward kept, as fp32 [1 or 2, rows, N]: words of the upper 16 bits, bytes below."""
    Np = (N + 15) // 16 * 16
    hi = kept[:, :2 * rows * Np].contiguous().view(torch.int16).view(-1, rows, Np).int() << 16
    lo = kept[:, 2 * rows * Np:].reshape(-1, rows, Np).int() << 8
    return (hi | lo)[..., :N].contiguous().view(torch.float32)


def check_forward(x, w, y, kept, act, bias=None, w_gate=None, bias_gate=None, residual=None):
    dt, K = x.dtype, x.shape[-1]
    X = x.double()

    def product(w, b):
        z = X @ w.double()
        tol = sums(K) * (X.abs() @ w.double().abs())
        if b is not None:
            z = z + b.double()
            tol = tol + 2.0 ** -23 * z.abs()
        return z, tol
    z, tz = product(w, bias)
    a, _ = act_of(z, act)
    ta = 1.13 * tz + 2.0 ** -20 * (z.abs() + 1) * (act != "none")
    if w_gate is not None:
        g, tg = product(w_gate, bias_gate)
        ta = ta * (g.abs() + tg) + a.abs() * tg + 2.0 ** -23 * (a * g).abs()
        a = a * g
    if residual is not None:
        a = a + residual.double()
        ta = ta + 2.0 ** -23 * a.abs()
    inside(y, a, rounded(a, ta, dt), "y")
    if kept is not None:
        # cut off after 24 bits: 2^-15 of the value at most
        k = unpacked(kept, X.shape[0], w.shape[1])
        inside(k[0], z, tz + 2.0 ** -15 * (z.abs() + tz), "z")
        if w_gate is not None:
            inside(k[1], g, tg + 2.0 ** -15 * (g.abs() + tg), "g")


def check_backward(dy, x, w, kept, grads, act, bias=None, w_gate=None, bias_gate=None):
    dt, (K, N), M = x.dtype, w.shape, x.numel() // x.shape[-1]
    D, X, W = dy.double().reshape(-1, N), x.double().reshape(-1, K), w.double()
    dx, dw, db, dwg, dbg = grads
    # of up to 2^16 elements what dz's rounding loses is multiplied as well: its rounding is what is left
    two = M * N <= 1 << 16
    e = step(dt) ** 2 if two else step(dt)
    parts = []  # (dz, what fp32 loses of it, weights, gradients)
    if act == "none" and w_gate is None:
        parts.append((D, torch.zeros_like(D), W, dw, db))
        e, two = 0.0, True
    else:
        k = unpacked(kept, M, N).double()
        z = k[0]
        a, slope = act_of(z, act)
        lost = 2.0 ** -19 * D.abs() * (z.abs() + 1) * (act != "none")
        if w_gate is None:
            parts.append((D * slope, lost, W, dw, db))
        else:
            g = k[1]
            parts.append((D * slope * g, lost * g.abs() + 2.0 ** -22 * (D * slope * g).abs(), W, dw,
                          db))
            parts.append((D * a, lost + 2.0 ** -23 * (D * a).abs(), w_gate.double(), dwg, dbg))
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    ref = sum(dz @ w.t() for dz, _, w, _, _ in parts)
    size = sum(dz.abs() @ w.abs().t() for dz, _, w, _, _ in parts)
    loss = sum((t + (tiny if e else 0)) @ w.abs().t() for _, t, w, _, _ in parts)

    def hold(got, ref, size, loss, n, name):
        tol = e * size * (1 + 2.0 ** -8) + loss * (1 + e) + sums(n) * size
        inside(got, ref, rounded(ref, tol, dt), name)
        rms = (1 if two else 2) * step(dt) / 3 ** 0.5 * ref.norm() + \
            ((sums(n) + (e if two else 0)) * size + loss).norm() + tiny * ref.numel() ** 0.5
        assert (got.double() - ref).norm() <= rms or ref.numel() < 1000, name

    if dx is not None:
        hold(dx.reshape(-1, K), ref, size, loss, N * len(parts), "dx")
    for i, (dz, t, _, dw, db) in enumerate(parts):
        if dw is not None:
            lost = X.abs().t() @ (t + (tiny if e else 0))
            hold(dw, X.t() @ dz, X.abs().t() @ dz.abs(), lost, M, f"dw{i}")
        if db is not None:
            # fp32 sums of M terms in any order: M 2^-24 of the terms' magnitudes at most
            r = dz.sum(0)
            inside(db, r, rounded(r, M * 2.0 ** -23 * dz.abs().sum(0) + t.sum(0), dt), f"db{i}")


def test_reference_slopes():
    """The derivatives above against central differences."""
    z = torch.linspace(-6, 6, 1201, dtype=torch.float64) + 1e-3
    for act in ACTS:
        up, down = act_of(z + 1e-5, act)[0], act_of(z - 1e-5, act)[0]
        assert ((up - down) / 2e-5 - act_of(z, act)[1]).abs().max() < 1e-8, act


def test_abi_refusals(L):
    at = 1 << 20  # never dereferenced: every call below is refused first

    def fwd(x=at, w=2 * at, wg=0, b=0, bg=0, r=0, y=3 * at, z=0, g=0, strides=(64, 64, 64, 64, 64),
            M=4, K=64, N=64, order=0, act=0, dtype=0, ws=64 * at, bytes=1 << 30):
        a = _FWD.pack(x, w, wg, b, bg, r, y, z, g, *strides, M, K, N, order, act, dtype)
        return L.dash_dense_fwd(a, ws, bytes, None)
    for bad in (dict(x=0), dict(w=0), dict(y=0), dict(M=0), dict(K=0), dict(N=-1), dict(order=2),
                dict(act=5), dict(act=-1), dict(dtype=3), dict(x=at + 1), dict(z=5 * at + 8), dict(bg=at), dict(g=at),
                dict(strides=(64, 64, 64, 64, 63)), dict(y=at), dict(y=2 * at), dict(y=64 * at),
                dict(z=3 * at), dict(b=3 * at), dict(r=3 * at, strides=(64, 64, 64, 72, 64)),
                dict(r=3 * at + 64)):
        assert fwd(**bad) == 1, bad
    assert fwd(dtype=2) == 2 and fwd(M=(1 << 31) - 1) == 2
    assert fwd(ws=0) == 5 and fwd(bytes=255) == 5 and fwd(ws=64 * at + 8) == 5
    assert L.dash_dense_fwd(None, at, 1 << 30, None) == 1
    assert L.dash_dense_fwd_workspace_bytes(None) == 0

    def bwd(dy=at, x=2 * at, w=3 * at, wg=0, z=0, g=0, dx=4 * at, dw=5 * at, dwg=0, db=0, dbg=0,
            strides=(64,) * 7, M=4, K=64, N=64, order=0, act=0, dtype=0, ws=64 * at, bytes=1 << 30):
        a = _BWD.pack(dy, x, w, wg, z, g, dx, dw, dwg, db, dbg, *strides, M, K, N, order, act, dtype)
        return L.dash_dense_bwd(a, ws, bytes, None)
    for bad in (dict(dy=0), dict(M=-1), dict(K=0), dict(N=0), dict(order=-1), dict(act=9),
                dict(dtype=7), dict(x=0), dict(w=0), dict(act=1), dict(g=at), dict(dwg=at),
                dict(dbg=at), dict(z=6 * at, g=7 * at), dict(z=6 * at, g=7 * at, wg=8 * at),
                dict(dx=at), dict(dw=2 * at), dict(dw=4 * at), dict(db=4 * at), dict(dw=5 * at + 1),
                dict(strides=(64, 64, 64, 64, 63, 64, 64)),
                dict(strides=(64, 64, 64, 64, 64, 63, 64))):
        assert bwd(**bad) == 1, bad
    assert bwd(dtype=2) == 2 and bwd(M=(1 << 31) - 1) == 2
    assert bwd(ws=0) == 5 and bwd(bytes=255) == 5
    assert L.dash_dense_bwd(None, at, 1 << 30, None) == 1


def test_workspace_sizes(L):
    """A part of the workspace for each operand that has to be copied, and for partial sums."""
    at = 1 << 20

    def need(x=at, w=2 * at, xs=64, ws=64, M=4, K=64, N=64, order=0):
        return L.dash_dense_fwd_workspace_bytes(
            _FWD.pack(x, w, 0, 0, 0, 0, 3 * at, 0, 0, xs, ws, 0, 0, N, M, K, N, order, 0, 0))
    assert need() == 256
    assert need(x=at + 2) == 256 + 4 * 128 and need(xs=65) == 256 + 4 * 128
    assert need(w=2 * at + 2) == 256 + 64 * 128 and need(ws=68) == 256 + 64 * 128
    assert need(K=7, xs=7) == 256 + 256  # 4 rows of 8, as a block of 256
    assert need(N=64, K=64, ws=70, order=1) == 256 + 64 * 128
    assert need(M=65, K=16384, N=256, xs=16384, ws=256) > 256 + 2 * 65 * 256 * 4
    assert need(M=64, K=16384, N=256, xs=16384, ws=256) == 256
    assert need(M=1, x=at, xs=3) == 256  # the stride of a single row has no meaning


# M, K, N: one row and element up; tile edges; odd; several tiles a CTA; long sums
SIZES = [(1, 1, 1), (1, 200, 2000), (16, 1000, 700), (64, 4096, 520), (65, 4096, 520), (48, 72, 24), (1, 64, 256), (3, 8, 40), (17, 200, 96), (129, 65, 130), (256, 64, 256),
         (257, 128, 513), (300, 1001, 77), (1, 4096, 1000), (33, 8192, 264), (1237, 96, 1000),
         (2100, 192, 8200)]
# what stands in the epilogue: act, bias, gate, residual
EPILOGUES = [("none", False, False, False), ("silu", False, True, False), ("gelu", True, False, True),
             ("gelu_tanh", True, True, True), ("relu", True, False, False)]


def case(M, K, N, order, dtype, epilogue, seed=0):
    act, b, g, r = epilogue
    x, w = make((M, K), dtype, seed), weight(K, N, order, dtype, seed + 1)
    a = dict(act=act, bias=make((N,), dtype, seed + 2, 0.5) if b else None,
             w_gate=weight(K, N, order, dtype, seed + 3) if g else None,
             bias_gate=make((N,), dtype, seed + 4, 0.5) if b and g else None)
    return x, w, a, make((M, N), dtype, seed + 5) if r else None


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("epilogue", EPILOGUES, ids=lambda e: e[0])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(L, size, epilogue, order, dtype):
    x, w, a, r = case(*size, order, dtype, epilogue)
    y, kept = dash.dense_fwd(x, w, residual=r, check=True, **a)
    check_forward(x, w, y, kept, residual=r, **a)
    assert (kept is None) == (a["act"] == "none" and a["w_gate"] is None)
    again, none = dash.dense_fwd(x, w, residual=r, keep=False, **a)
    assert none is None and torch.equal(again, y)


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("epilogue", EPILOGUES, ids=lambda e: e[0])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(L, size, epilogue, order, dtype):
    M, K, N = size
    x, w, a, r = case(*size, order, dtype, epilogue)
    _, kept = dash.dense_fwd(x, w, **a)
    dy = make((M, N), dtype, 9)
    grads = dash.dense_bwd(dy, x, w, kept, check=True, **a)
    assert grads[1].stride() == w.stride() or 1 in (K, N)
    check_backward(dy, x, w, kept, grads, **a)
    again = dash.dense_bwd(dy, x, w, kept, **a)
    assert all(p is q or torch.equal(p, q) for p, q in zip(grads, again))
    dx = dash.dense_bwd(dy, x, w, kept, need_dw=False, **a)
    assert torch.equal(dx[0], grads[0]) and dx[1] is None and dx[3] is None
    dw = dash.dense_bwd(dy, x, w, kept, need_dx=False, **a)
    assert dw[0] is None and torch.equal(dw[1], grads[1])


@gpu
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("order", ["kn", "nk"])
def test_views(L, order, offset):
    """Rows at wider strides, off 16 bytes too, outputs into views whose surroundings stay."""
    M, K, N, dt = 137, 72, 136, BF
    x, w, a, r = case(M, K, N, order, dt, ("silu", True, True, True))
    dy = make((M, N), dt, 9)
    y, kept = dash.dense_fwd(x, w, residual=r, **a)
    grads = dash.dense_bwd(dy, x, w, kept, **a)

    def wide(t):
        big = torch.full((t.shape[0] + 2, t.shape[1] + 24), 7.0, dtype=dt, device="cuda")
        v = big[1:-1, offset:offset + t.shape[1]]
        v.copy_(t)
        return big, v

    def wide_w(t):
        big, v = wide(t if order == "kn" else t.t())
        return big, v if order == "kn" else v.t()
    xv, rv, dv = wide(x)[1], wide(r)[1], wide(dy)[1]
    wv = wide_w(w)[1]
    a["w_gate"] = wide_w(a["w_gate"])[1]
    big, out = wide(torch.zeros_like(y))
    got, kept2 = dash.dense_fwd(xv, wv, residual=rv, out=out, check=True, **a)
    assert got is out and torch.equal(out, y)
    assert torch.equal(unpacked(kept2, M, N), unpacked(kept, M, N))
    assert (big == 7).sum() == big.numel() - out.numel() + (out == 7).sum()
    bx, dx = wide(torch.zeros_like(x))
    bw, dw = wide_w(torch.zeros_like(w))
    bg, dg = wide_w(torch.zeros_like(w))
    res = dash.dense_bwd(dv, xv, wv, kept, dx=dx, dw=dw, dw_gate=dg, **a)
    assert res[0] is dx and res[1] is dw and res[3] is dg
    assert all(torch.equal(p, q) for p, q in zip(res, grads))
    for b, o in ((bx, dx), (bw, dw), (bg, dg)):
        assert (b == 7).sum() == b.numel() - o.numel() + (o == 7).sum()
    # a workspace of the size that is named serves, one that is smaller is refused
    need = dash.dense_fwd_workspace_bytes(xv, wv, w_gate=a["w_gate"], residual=rv, out=out)
    need2 = dash.dense_bwd_workspace_bytes(dv, xv, wv, kept, dx=dx, dw=dw, dw_gate=dg, **a)
    for n, n2 in ((need, need2), (need - 1, need2 - 1)):
        ws, ws2 = (torch.empty(m, dtype=torch.uint8, device="cuda") for m in (n, n2))
        if n == need:
            dash.dense_fwd(xv, wv, residual=rv, out=out, workspace=ws, **a)
            dash.dense_bwd(dv, xv, wv, kept, dx=dx, dw=dw, dw_gate=dg, workspace=ws2, **a)
            assert torch.equal(out, y) and torch.equal(dx, grads[0]) and torch.equal(dg, grads[3])
            continue
        with pytest.raises(ValueError):
            dash.dense_fwd(xv, wv, residual=rv, out=out, workspace=ws, **a)
        with pytest.raises(ValueError):
            dash.dense_bwd(dv, xv, wv, kept, dx=dx, dw=dw, dw_gate=dg, workspace=ws2, **a)
    # onto the residual stream itself, from rows of a [B, S, K] tensor, one row for all
    same = r.clone()
    dash.dense_fwd(x, w, residual=same, out=same, **a)
    assert torch.equal(same, y)
    x3 = x[:136].view(2, 68, K).transpose(0, 1).contiguous().transpose(0, 1)
    y3 = dash.dense_fwd(x[:136].view(2, 68, K), w, **a)[0]
    with pytest.raises(ValueError):
        dash.dense_fwd(x3, w, **a)
    assert y3.shape == (2, 68, N)
    one = dash.dense_bwd(dy[:1].expand(M, N), x, w, kept, **a)
    ref = dash.dense_bwd(dy[:1].repeat(M, 1), x, w, kept, **a)
    assert all(torch.equal(p, q) for p, q in zip(one, ref))


@gpu
def test_no_rows(L):
    x, w, a, _ = case(1, 40, 24, "kn", BF, ("gelu", True, True, False))
    x, dy = x[:0], torch.empty(0, 24, dtype=BF, device="cuda")
    y, kept = dash.dense_fwd(x, w, **a)
    assert y.shape == (0, 24) and kept.shape == (2, 0)
    dx, *rest = dash.dense_bwd(dy, x, w, kept, **a)
    assert dx.shape == (0, 40) and all((t == 0).all() for t in rest)


@gpu
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_special_values_stay_in_their_row(L, bad):
    """A row of x that is not finite spoils its own row of y and dx only; a split long sum too."""
    for M, K, N in ((300, 72, 200), (2, 8192, 64), (70, 8192, 64)):
        x, w, a, _ = case(M, K, N, "kn", BF, ("silu", False, True, False))
        y, kept = dash.dense_fwd(x, w, **a)
        dy = make((M, N), BF, 3)
        dx = dash.dense_bwd(dy, x, w, kept, need_dw=False, **a)[0]
        x[M // 2, K - 1] = bad
        y2, _ = dash.dense_fwd(x, w, **a)
        assert not y2[M // 2].isfinite().any()
        y2[M // 2] = y[M // 2]
        assert torch.equal(y2, y)
        dy[M // 2, 5] = bad
        dx2 = dash.dense_bwd(dy, x, w, kept, need_dw=False, **a)[0]
        assert not dx2[M // 2].isfinite().any()
        dx2[M // 2] = dx[M // 2]
        assert torch.equal(dx2, dx)


@gpu
def test_activations_at_the_ends(L):
    """Far arguments: the activations and their slopes go to 0 and 1, without NaN."""
    z = torch.tensor([[-3e30, -200.0, -90.0, -30.0, -1e-4, 0.0, 1e-4, 30.0, 90.0, 3e30]], dtype=BF,
                     device="cuda")
    eye = torch.eye(10, dtype=BF, device="cuda")
    for act in ACTS:
        y, kept = dash.dense_fwd(z, eye, act=act)
        check_forward(z, eye, y, kept, act)
        dx, dw, *_ = dash.dense_bwd(torch.ones_like(z), z, eye, kept, act=act)
        # (at 64 bits the ends lie inside the range: slopes of 0 and 1 there)
        slope = act_of(z.double().clamp(-3e4, 3e4), act)[1]
        assert torch.allclose(dx.double(), slope, atol=2.0 ** -8, rtol=2.0 ** -8)
        assert dx.isfinite().all() and dw.isfinite().all()


@gpu
def test_streams_graphs_and_workspaces(L):
    """On another stream, into captured graphs (replayed with new inputs), workspaces handed in."""
    M, K, N = 200, 1024, 320
    x, w, a, r = case(M, K, N, "kn", BF, ("silu", False, True, True))
    dy = make((M, N), BF, 9)
    ref = dash.dense_fwd(x, w, residual=r, **a)
    want = dash.dense_bwd(dy, x, w, ref[1], **a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, kept = dash.dense_fwd(x, w, residual=r, stream=s, **a)
    got = dash.dense_bwd(dy, x, w, kept, stream=s, **a)
    s.synchronize()
    assert torch.equal(y, ref[0])
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, want))
    ws1 = torch.empty(dash.dense_fwd_workspace_bytes(x, w, w_gate=a["w_gate"]), dtype=torch.uint8,
                      device="cuda").fill_(255)
    ws2 = torch.empty(dash.dense_bwd_workspace_bytes(dy, x, w, kept, **a), dtype=torch.uint8,
                      device="cuda").fill_(255)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, kept = dash.dense_fwd(x, w, residual=r, workspace=ws1, **a)
        got = dash.dense_bwd(dy, x, w, kept, workspace=ws2, **a)
    for seed in (20, 21):
        x.copy_(make((M, K), BF, seed))
        dy.copy_(make((M, N), BF, seed + 5))
        g.replay()
        y1, k1 = dash.dense_fwd(x, w, residual=r, **a)
        assert torch.equal(y, y1) and torch.equal(unpacked(kept, M, N), unpacked(k1, M, N))
        assert all(p is q or torch.equal(p, q)
                   for p, q in zip(got, dash.dense_bwd(dy, x, w, k1, **a)))
    dash.status(ws1), dash.status(ws2)


@gpu
def test_refusals(L):
    x, w, a, r = case(4, 64, 32, "kn", BF, ("silu", True, True, True))
    _, kept = dash.dense_fwd(x, w, **a)
    dy = make((4, 32), BF, 9)
    for bad in (lambda: dash.dense_fwd(x.cpu(), w), lambda: dash.dense_fwd(x.float(), w.float()),
                lambda: dash.dense_fwd(x, w.half()), lambda: dash.dense_fwd(x, w[:63]),
                lambda: dash.dense_fwd(x, w, act="tanh"), lambda: dash.dense_fwd(x, w, w[0, :31]),
                lambda: dash.dense_fwd(x, w, residual=x), lambda: dash.dense_fwd(x, w, out=dy[:3]),
                lambda: dash.dense_fwd(x, w[::2, ::2].contiguous()),
                lambda: dash.dense_fwd(x[:, ::2], w[:32]), lambda: dash.dense_fwd(x[:, :32], w[::2, ::2]),
                lambda: dash.dense_fwd(x, w, w_gate=w.t().contiguous().t()),
                lambda: dash.dense_fwd(x, w, bias_gate=a["bias"]),
                lambda: dash.dense_fwd(x, w, out=dy[:1].expand(4, 32)),
                lambda: dash.dense_fwd(x, w, workspace=torch.empty(8, device="cuda")),
                lambda: dash.dense_fwd(x, w[:, :0]), lambda: dash.dense_fwd(x[:, :0], w[:0]),
                lambda: dash.dense_bwd(dy, x, w, act="silu"),
                lambda: dash.dense_bwd(dy, x, w, kept[:1], act="silu", w_gate=w),
                lambda: dash.dense_bwd(dy, x, w, kept, act="silu"),
                lambda: dash.dense_bwd(dy, x, w, kept.char(), act="silu", w_gate=w),
                lambda: dash.dense_bwd(dy[:3], x, w), lambda: dash.dense_bwd(dy, x, w, dw_gate=w),
                lambda: dash.dense_bwd(dy, x, w, dw=torch.empty_like(w).t().contiguous().t()),
                lambda: dash.dense_bwd(dy.half(), x, w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dash.dense_fwd(x, w, residual=dy, out=w[:4]),
                lambda: dash.dense_fwd(x[:2], w, out=r[:2], bias=r[1]),
                lambda: dash.dense_bwd(dy, x, w, dx=x), lambda: dash.dense_bwd(dy, x, w, dw=w)):
        with pytest.raises(dash.DashError):
            bad()


@gpu
@pytest.mark.parametrize("M", [700, 5])
def test_failure_detection(L, M):
    """Loads that end early: the waits for them run out, the call is reported, the next one is right."""
    M, K, N = M, 640, 1000
    x, w, a, r = case(M, K, N, "nk", BF, ("gelu", True, False, True))
    y, _ = dash.dense_fwd(x, w, residual=r, **a)
    limit = dash.wait_limit()
    dash.set_wait_limit(0.2)
    try:
        for block in (0, 1):
            assert L.dash_dense_withhold(block) == 0
            with pytest.raises(dash.DashError) as e:
                dash.dense_fwd(x, w, residual=r, check=True, **a)
            assert e.value.code == 4
    finally:
        L.dash_dense_withhold(-1)
        dash.set_wait_limit(limit)
    again, _ = dash.dense_fwd(x, w, residual=r, check=True, **a)
    assert torch.equal(again, y)


@gpu
@pytest.mark.parametrize("size", [(1, 8192, 129), (1, 16384, 4), (3, 8192, 130), (2, 4096, 259)], ids=str)
def test_few_rows_whose_outputs_do_not_fill_a_warp(L, size):
    """A CTA of a cluster finishes a part of the outputs that is no whole number of warps, some lanes of
    it behind the last column; they meet again at the cluster's barrier."""
    x, w, a, r = case(*size, "kn", BF, ("silu", True, True, True))
    y, kept = dash.dense_fwd(x, w, residual=r, check=True, **a)
    check_forward(x, w, y, kept, residual=r, **a)
    for _ in range(20):
        assert torch.equal(dash.dense_fwd(x, w, residual=r, check=True, **a)[0], y)


@gpu
@pytest.mark.parametrize("M,block", [(700, 7), (5, 13)])
def test_failure_behind_the_first_filling(L, M, block):
    """The loads end when every place of a ring has been filled once: nothing of the call is under way
    any more when the next ones, which use the same shared memory, give their usual bits."""
    K, N = 8192, 1000
    x, w, a, r = case(M, K, N, "nk", BF, ("silu", False, True, True))
    y, kept = dash.dense_fwd(x, w, residual=r, **a)
    dy = make((M, N), BF, 9)
    grads = dash.dense_bwd(dy, x, w, kept, **a)
    limit = dash.wait_limit()
    dash.set_wait_limit(0.05)
    try:
        assert L.dash_dense_withhold(block) == 0
        with pytest.raises(dash.DashError) as e:
            dash.dense_fwd(x, w, residual=r, check=True, **a)
        assert e.value.code == 4
        L.dash_dense_withhold(0)
        with pytest.raises(dash.DashError) as e:
            dash.dense_bwd(dy, x, w, kept, check=True, **a)
        assert e.value.code == 4
    finally:
        L.dash_dense_withhold(-1)
        dash.set_wait_limit(limit)
    for _ in range(3):
        assert torch.equal(dash.dense_fwd(x, w, residual=r, check=True, **a)[0], y)
        again = dash.dense_bwd(dy, x, w, kept, check=True, **a)
        assert all(p is q or torch.equal(p, q) for p, q in zip(grads, again))


@gpu
@pytest.mark.parametrize("epilogue", [EPILOGUES[0], EPILOGUES[1], EPILOGUES[3]], ids=lambda e: e[0])
@pytest.mark.parametrize("size", [(127, 300, 512), (128, 4099, 512), (129, 300, 500), (2, 155648, 24),
                                  (2, 155649, 24), (1, 520, 20000)], ids=str)
def test_backward_of_few_rows(L, size, epilogue):
    """The second term of dz in a tile's other half, and where it does not fit there."""
    M, K, N = size
    x, w, a, r = case(*size, "nk", BF, epilogue)
    _, kept = dash.dense_fwd(x, w, **a)
    dy = make((M, N), BF, 9)
    grads = dash.dense_bwd(dy, x, w, kept, check=True, **a)
    check_backward(dy, x, w, kept, grads, **a)
    need = dash.dense_bwd_workspace_bytes(dy, x, w, kept, **a)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    again = dash.dense_bwd(dy, x, w, kept, workspace=ws[:need], check=True, **a)
    assert all(p is q or torch.equal(p, q) for p, q in zip(grads, again))
    assert (ws[need:] == 255).all()


@gpu
def test_the_second_term_reads_the_weights_once(L):
    """dx of few rows with and without an activation: of weights that L2 does not hold (268 MB, 40 us of
    memory) a second pass would take half as long again and more."""
    M, K, N = 8, 16384, 8192
    x, w, dy = make((M, K), BF, 0), make((K, N), BF, 1, K ** -0.5), make((M, N), BF, 2)
    _, kept = dash.dense_fwd(x, w, act="relu")
    time = {}
    for act in ("none", "relu"):
        dash.dense_bwd(dy, x, w, kept, act=act, need_dw=False)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                dash.dense_bwd(dy, x, w, kept, act=act, need_dw=False)
        runs = []
        for _ in range(12):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            g.replay()
            end.record()
            end.synchronize()
            runs.append(start.elapsed_time(end))
        time[act] = sorted(runs)[len(runs) // 2]
    assert time["relu"] < 1.3 * time["none"], time


@gpu
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("size", [(64, 64, 64), (64, 96, 1000), (200, 300, 300), (2000, 72, 24), (300, 72, 400)],
                         ids=str)
def test_infinities_in_the_backwards_operands(L, size, order):
    """An infinity in x or in a weight is multiplied by dz: what comes out is infinite or NaN as dz's signs
    and zeros have it, whether dz goes in one term or in two.  (relu, and dy of few bits: dz fits 16 bits,
    so that a second term is 0.)"""
    M, K, N = size
    x, w, a, _ = case(M, K, N, order, BF, ("relu", False, False, False))
    dy = make((M, N), BF, 9).sign() + 0.25
    dy[:, N // 2] = 0.0
    y, kept = dash.dense_fwd(x, w, act="relu")
    dz = dy.double() * (unpacked(kept, M, N)[0] > 0)
    assert (dz == dz.to(BF).double()).all()
    x[M // 2, 3], x[M // 3, K - 1] = math.inf, -math.inf
    w = w.clone(memory_format=torch.preserve_format)
    w[5, N // 3], w[K - 2, N - 1], w[7, N // 2] = -math.inf, math.inf, math.inf
    dx, dw, *_ = dash.dense_bwd(dy, x, w, kept, act="relu")
    for got, ref in ((dx, dz @ w.double().t()), (dw, x.double().t() @ dz)):
        got = got.double()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.isinf(), ref.isinf())
        assert torch.equal(got[ref.isinf()], ref[ref.isinf()])
        assert ref.isinf().any()


def test_abi_terms(L):
    at = 1 << 20  # never dereferenced: every call below is refused first

    def bwd(terms, M=4, act=1, ws=0):
        a = _BWD.pack(at, 2 * at, 3 * at, 0, 6 * at, 0, 4 * at, 5 * at, 0, 0, 0, *(64,) * 7, M, 64, 64, 0,
                      act, 0)
        need = L.dash_dense_bwd_terms_workspace_bytes(a, terms)
        return L.dash_dense_bwd_terms(a, terms, ws, 0, None), need
    assert bwd(-1) == (1, 0) and bwd(3) == (1, 0)
    code, one = bwd(1)
    assert code == 5 and bwd(2)[1] > one and bwd(0) == bwd(2)
    assert bwd(0, M=1025) == bwd(1, M=1025) and bwd(2, M=1025)[1] > bwd(1, M=1025)[1]
    assert bwd(2, act=0) == bwd(1, act=0)
    assert bwd(2, M=(1 << 29) + 1) == (2, 0) and bwd(1, M=(1 << 29) + 1)[0] == 5


@gpu
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("epilogue", EPILOGUES[1:], ids=lambda e: e[0])
@pytest.mark.parametrize("size", [(48, 72, 24), (300, 1001, 277), (700, 264, 1000)], ids=str)
def test_terms(L, size, epilogue, order):
    """One term or two as the caller has it, at sizes on both sides of the default's."""
    M, K, N = size
    x, w, a, _ = case(*size, order, BF, epilogue)
    _, kept = dash.dense_fwd(x, w, **a)
    dy = make((M, N), BF, 9)
    default, one, two = (dash.dense_bwd(dy, x, w, kept, terms=t, check=True, **a) for t in (None, 1, 2))
    same = two if M * N <= 1 << 16 else one
    assert all(p is q or torch.equal(p, q) for p, q in zip(default, same))
    # (relu without a gate: dz is dy or 0, which 16 bits hold)
    exact = epilogue[0] == "relu"
    assert torch.equal(one[1], two[1]) == exact and torch.equal(one[0], two[0]) == exact
    # in the norm: two terms leave the results' own rounding (as for few elements above)
    k = unpacked(kept, M, N).double()
    act, slope = act_of(k[0], a["act"])
    parts = [(dy.double() * slope * (k[1] if len(k) > 1 else 1.0), w.double(), 1)]
    if len(k) > 1:
        parts.append((dy.double() * act, a["w_gate"].double(), 3))
    e, X = step(BF), x.double()

    def hold(got, ref, size, n):
        lost = (sums(n) + e * e + 2.0 ** -17) * size.norm()
        assert (got.double() - ref).norm() <= e / 3 ** 0.5 * ref.norm() + lost or ref.numel() < 1000
    hold(two[0], sum(d @ u.t() for d, u, _ in parts), sum(d.abs() @ u.abs().t() for d, u, _ in parts),
         N * len(parts))
    for d, _, i in parts:
        hold(two[i], X.t() @ d, X.abs().t() @ d.abs(), M)
    need = dash.dense_bwd_workspace_bytes(dy, x, w, kept, terms=2, **a)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    again = dash.dense_bwd(dy, x, w, kept, terms=2, workspace=ws, check=True, **a)
    assert all(p is q or torch.equal(p, q) for p, q in zip(two, again))
    for bad in (0, 3, "2"):
        with pytest.raises(ValueError):
            dash.dense_bwd(dy, x, w, kept, terms=bad, **a)


@gpu
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("size", [(100, 200, 300), (700, 264, 1000), (2500, 72, 4099)], ids=str)
def test_special_values_of_two_terms(L, size, order):
    """Infinities and NaN in any operand, with dz that two terms are needed for: one term's where one term
    has them, two terms' bits elsewhere."""
    M, K, N = size
    x, w, a, _ = case(*size, order, BF, EPILOGUES[1])
    _, kept = dash.dense_fwd(x, w, **a)
    dy = make((M, N), BF, 9)
    clean = dash.dense_bwd(dy, x, w, kept, terms=2, **a)
    w, a["w_gate"] = (t.clone(memory_format=torch.preserve_format) for t in (w, a["w_gate"]))
    x[M // 2, 3], x[M // 3, K - 1], x[M // 3, K // 2] = math.inf, -math.inf, math.nan
    w[5, N // 3], a["w_gate"][K - 2, N - 1] = -math.inf, math.inf
    for step_ in range(2):
        one, two = (dash.dense_bwd(dy, x, w, kept, terms=t, **a) for t in (1, 2))
        for i in (0, 1, 3):
            bad = ~one[i].isfinite()
            assert bad.any() and one[i].isinf().any() and not bad.all()
            assert torch.equal(two[i].isnan(), one[i].isnan())
            inf = one[i].isinf()
            assert torch.equal(two[i][inf], one[i][inf])
            assert torch.equal(two[i][~bad], clean[i][~bad]) or step_
        dy[M // 4, N // 2] = math.inf


@gpu
@pytest.mark.parametrize("size", [(200, 1, 64), (3, 1, 77), (70, 128, 300)], ids=str)
def test_what_is_kept_is_rounded(L, size):
    """z and g in 24 bits are off by half a step at most, 2^-16, and as often up as down.  Of one product
    and a bias z itself is off by 2^-24 of its parts; of a hundred and more what the sums are off is small
    in the mean."""
    M, K, N = size
    x, w, a, _ = case(*size, "kn", BF, EPILOGUES[3])
    y, kept = dash.dense_fwd(x, w, **a)
    k = unpacked(kept, M, N).double()
    for got, u, b in zip(k, (w, a["w_gate"]), (a["bias"], a["bias_gate"])):
        p = x.double() @ u.double()
        z = p + b.double()
        own = sums(K) * (x.double().abs() @ u.double().abs()) if K > 1 else 0.0
        own = own + 2.0 ** -24 * (p.abs() + b.double().abs() + z.abs())
        assert ((got - z).abs() <= 2.0 ** -16 * (z.abs() + own) + own).all()
        # an error spread evenly over a step of 2^-15 has a mean of 0 and a deviation of 2^-15 / sqrt 12
        # of the value's power of two: five deviations of the mean
        up = ((got - z) * z.sign() / 2.0 ** z.abs().log2().floor()).mean()
        assert up.abs() <= 5 * 2.0 ** -15 / 12 ** 0.5 / z.numel() ** 0.5 + 2.0 ** -22


@gpu
def test_special_values_are_kept(L):
    x = torch.tensor([[math.nan, math.inf, -math.inf, 3.38e38, -0.0, 1e-38]], dtype=BF, device="cuda").t()
    one = torch.ones(1, 16, dtype=BF, device="cuda")
    _, kept = dash.dense_fwd(x.contiguous(), one, act="silu")
    z = unpacked(kept, 6, 16)[0, :, 0]
    assert z[0].isnan() and z[1] == math.inf and z[2] == -math.inf and z[4] == 0
    assert z[3] == x[3, 0].float() and abs(z[5] - x[5, 0].float()) <= 2.0 ** -16 * 1e-38


@gpu
@pytest.mark.parametrize("size", [(40, 256, 300), (300, 264, 200)], ids=str)
def test_special_values_come_and_go_in_a_captured_backward(L, size):
    """What flags a sum that is not finite is cleared by every call: replays with and without infinities, and
    two graphs that share a workspace, one after the other."""
    M, K, N = size
    x, w, a, _ = case(*size, "kn", BF, EPILOGUES[1])
    _, kept = dash.dense_fwd(x, w, **a)
    dys = [make((M, N), BF, s) for s in (9, 10)]
    clean = [dash.dense_bwd(dy, x, w, kept, **a) for dy in dys]
    ws = torch.full((dash.dense_bwd_workspace_bytes(dys[0], x, w, kept, **a),), 255, dtype=torch.uint8,
                    device="cuda")
    graphs, outs = [], []
    for dy in dys:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dash.dense_bwd(dy, x, w, kept, workspace=ws, **a))
        graphs.append(g)
    good = x[1, 2].clone()
    for bad in (math.inf, 0.0, math.inf, math.nan, 0.0):
        x[1, 2] = bad if bad else good
        for g, dy, out, ref in zip(graphs, dys, outs, clean):
            g.replay()
            if not bad:
                assert all(p is q or torch.equal(p, q) for p, q in zip(out, ref))
                continue
            one = dash.dense_bwd(dy, x, w, kept, terms=1, **a)
            for i in (0, 1, 3):
                assert torch.equal(out[i].isnan(), one[i].isnan())
                assert torch.equal(out[i].isinf(), one[i].isinf())
            assert not out[1][2].isfinite().any() and torch.equal(out[1][3], ref[1][3])
    dash.status(ws)
