"""Row norms and the residual join against their definitions in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32.  A row sum adds at most 100 terms one after
another per thread and 21 levels of partial sums, so a sum of n terms t is off by at most 128 u
sum |t|; rstd (half of that, relative) and every product add a few u.  Each bound below is
2^-16 = 256 u times the sum of the absolute values of the terms that make up a value, formed
with the same formulas; the column sums of the weight gradients add their rows in at most 100
terms one after another and 33 partial sums.  An output of a narrower type is off by half a
step more: eps / 2 relative to the value."""
import ctypes

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build, norms

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def near(name, got, ref, terms, extra=0.0):
    tol = 2.0 ** -16 * terms + extra
    if got.dtype != F32:
        f = torch.finfo(got.dtype)
        tol = tol + f.eps / 2 * (ref.abs() + tol) + f.smallest_normal * f.eps
    else:
        tol = tol + 2.0 ** -24 * ref.abs() + 2.0 ** -140
    err = (got.double() - ref).abs()
    assert got.shape == ref.shape and (err <= tol).all(), (name, (err - tol).max().item())


def gates(gate, x):
    """The gate's row for every row of x, or ones."""
    if gate is None:
        return torch.ones_like(x).double()
    g = gate.double().reshape(-1, x.shape[-1])
    rows = x.numel() // x.shape[-1]
    return g.repeat_interleave(rows // g.shape[0], 0).view(x.shape)


def forward(x, a, w_post, gate, w_next, skip, branch):
    """y, h, rstd_a, rstd_y in 64 bits and the sums of absolute terms of y and h."""
    x, a = x.double(), a.double()
    ra = (a.square().mean(-1, keepdim=True) + EPS).rsqrt() if w_post is not None else 1.0
    t = branch * gates(gate, x) * a * ra * (w_post.double() if w_post is not None else 1.0)
    y = skip * x + t
    ty = (skip * x).abs() + t.abs()
    if w_next is None:
        return y, None, ra, None, ty, None
    ry = (y.square().mean(-1, keepdim=True) + EPS).rsqrt()
    w = w_next.double()
    # rstd_y is off by what y is: sum |y| ty / sum y^2, relative
    spread = 1.0 + (y.abs() * ty).mean(-1, keepdim=True) * ry ** 2
    return y, y * ry * w, ra, ry, ty, (ty + y.abs() * spread) * ry * w.abs()


def backward(dy, dh, y, a, ra, ry, w_post, gate, w_next, skip, branch):
    """The gradients in 64 bits from the rows and rstd given, each with its absolute terms."""
    g, a = gates(gate, a), a.double()
    D = dy.double() if dy is not None else torch.zeros_like(a)
    Dt = D.abs()
    out = {}
    if w_next is not None:
        q, w, dh = y.double() * ry, w_next.double(), dh.double()
        D = D + ry * (dh * w - q * (dh * w * q).mean(-1, keepdim=True))
        Dt = Dt + ry * ((dh * w).abs() + q.abs() * (dh * w * q).abs().mean(-1, keepdim=True))
        rows = tuple(range(a.dim() - 1))
        out["dw_next"] = (dh * q).sum(rows), (dh * q).abs().sum(rows)
    out["dx"] = skip * D, abs(skip) * Dt
    z = a * ra
    wp = w_post.double() if w_post is not None else torch.ones(a.shape[-1]).double().to(a.device)
    t, tt = branch * g * D, (branch * g).abs() * Dt
    if w_post is not None:
        out["dw_post"] = (t * z).flatten(0, -2).sum(0), (tt * z.abs()).flatten(0, -2).sum(0)
        u, ut = t * wp, tt * wp.abs()
        out["da"] = (ra * (u - z * (u * z).mean(-1, keepdim=True)),
                     ra * (ut + z.abs() * (ut * z.abs()).mean(-1, keepdim=True)))
    else:
        out["da"] = t, tt
    if gate is not None:
        n = gate.numel() // gate.shape[-1]
        d, dt = branch * D * wp * z, abs(branch) * Dt * (wp * z).abs()
        out["dgate"] = tuple(v.reshape(n, -1, gate.shape[-1]).sum(1).view(gate.shape)
                             for v in (d, dt))
    return out


def make(shape, dtype, seed, by=1.0, plus=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * by + plus).to(dtype)


def run_join(shape, dtype, wdtype, gate, post=True, nxt=True, use_dy=True, skip=0.9, branch=-0.6):
    C = shape[-1]
    x, a = make(shape, dtype, 1, 2.0), make(shape, dtype, 2, 0.5)
    wp = make((C,), wdtype, 3, 0.2, 1.0) if post else None
    wn = make((C,), wdtype, 4, 0.2, 1.0) if nxt else None
    g = None if gate is None else make(gate, wdtype, 5, 0.5, 0.3)
    w = dict(w_post=wp, gate=g, w_next=wn)
    s = dict(skip_scale=skip, branch_scale=branch)
    y, h, ra, ry = dash.join_fwd(x, a, **w, **s, eps=EPS)
    Y, H, RA, RY, ty, th = forward(x, a, wp, g, wn, skip, branch)
    near("y", y, Y, ty)
    if nxt:
        near("h", h, H, th)
        near("rstd_y", ry, RY[..., 0], (RY * (th / H.abs().clamp_min(1e-30)).amin(-1, keepdim=True))[..., 0])
    else:
        assert h is None and ry is None
    if post:
        near("rstd_a", ra, RA[..., 0], RA[..., 0])
    dy = make(shape, dtype, 6) if use_dy else None
    dh = make(shape, dtype, 7) if nxt else None
    got = dict(zip(("dx", "da", "dw_post", "dgate", "dw_next"),
                   dash.join_bwd(dy, dh, y, a, ra, ry, **w, **s)))
    want = backward(dy, dh, y, a, ra.double()[..., None] if post else 1.0,
                    ry.double()[..., None] if nxt else None, wp, g, wn, skip, branch)
    for n, t in got.items():
        if n not in want:
            assert t is None, n
        else:
            near(n, t, *want[n])
    return got


WIDTHS = [1, 2, 5, 31, 64, 100, 128, 264, 512, 1001, 1024, 2040, 2048, 4096, 4104, 8192, 8200,
          16384, 16385, 16392, 40000]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("C", WIDTHS)
def test_join_widths(L, C, dtype):
    run_join((2, 5, C), dtype, dtype, (2, C))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape,gate", [
    ((1, 96), None), ((1, 96), (96,)), ((1, 96), (1, 96)), ((1, 4096), (4096,)),
    ((700, 96), (96,)), ((700, 1031), (1031,)), ((3, 300, 256), (3, 256)),
    ((17, 9, 512), (17, 512)), ((33, 5, 128), (33, 128)), ((400, 3, 72), (400, 72)),
    ((2, 31, 264), (2, 31, 264)),       # every row its own gate
    ((2, 31, 2056), (2, 31, 2056)), ((3000, 64), (64,)), ((0, 64), (64,)), ((2, 0, 64), None)], ids=str)
def test_join_rows_and_gates(L, shape, gate, dtype):
    run_join(shape, dtype, dtype, gate)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 130, 3000, 17000])
@pytest.mark.parametrize("post,nxt,use_dy,gated", [(False, True, True, True), (True, False, True, True),
                                                   (False, False, True, False),
                                                   (True, True, False, False),
                                                   (False, True, False, True)])
def test_join_without_some_parts(L, post, nxt, use_dy, gated, C):
    run_join((3, 11, C), BF, BF, (3, C) if gated else None, post, nxt, use_dy)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("C", [72, 130, 2048, 20000])
def test_join_fp32_weights(L, C, dtype):
    got = run_join((4, 7, C), dtype, F32, (4, C))
    assert got["dw_post"].dtype == got["dgate"].dtype == got["dw_next"].dtype == F32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("shape", [(1, 1), (3, 40, 128), (2, 100, 1001), (5, 4096), (2, 20000),
                                   (60000, 128)], ids=str)
@pytest.mark.parametrize("res", [False, True])
def test_norm(L, shape, dtype, res):
    x, w = make(shape, dtype, 1, 3.0), make(shape[-1:], dtype, 2, 0.2, 1.0)
    h, rstd = dash.norm_fwd(x, w, eps=EPS)
    zero = torch.zeros_like(x)
    Y, H, _, RY, ty, th = forward(x, zero, None, None, w, 1.0, 1.0)
    near("h", h, H, th)
    near("rstd", rstd, RY[..., 0], 2 * RY[..., 0])
    dh, dres = make(shape, dtype, 3), make(shape, dtype, 4) if res else None
    dx, dw = dash.norm_bwd(dh, x, rstd, w, dres=dres)
    want = backward(dres, dh, x, zero, 1.0, rstd.double()[..., None], None, None, w, 1.0, 1.0)
    near("dx", dx, *want["dx"])
    near("dw", dw, *want["dw_next"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("C", [17, 33, 65, 126, 250, 270, 499, 1001, 1503, 2052, 2731, 5003, 12271,
                               16361])
def test_rows_off_the_grid(L, C, dtype):
    """Enough rows of a length that 16 bytes do not divide, gated per sequence."""
    run_join((2, 70, C), dtype, dtype, (2, C))


@pytest.mark.gpu
@pytest.mark.parametrize("shape,gate,wdtype", [((2, 70, 1001), (2, 70, 1001), BF),  # own gates
                                               ((131, 257), (257,), F32), ((9, 8, 99), (9, 99), F32),
                                               ((3000, 65), None, BF), ((1, 66, 4099), (4099,), BF)],
                         ids=str)
def test_rows_off_the_grid_gates(L, shape, gate, wdtype):
    run_join(shape, BF, wdtype, gate)
    run_join(shape, BF, wdtype, gate, post=False, use_dy=False)
    run_join(shape, BF, wdtype, gate, nxt=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,C,offset,stride,weights", [
    (90, 251, 3, 251, 0), (90, 251, 3, 258, 1), (90, 256, 1, 256, 0), (90, 256, 0, 261, 0),
    (90, 256, 0, 256, 1), (77, 1030, 5, 1036, 3), (77, 64, 7, 71, 0), (70, 9000, 1, 9003, 1)])
@pytest.mark.parametrize("alike", [True, False])
def test_rows_off_the_grid_lie(L, dtype, rows, C, offset, stride, weights, alike):
    """Rows at any offset and stride, the same for all tensors or not, NaN in everything around
    them: the outputs are right and what lies around them stays."""
    def lay(t, k=0):  # t's rows at the offset and stride, in a buffer of NaN
        if not alike:
            k *= 2
        else:
            k = 0
        buf = torch.full((offset + k + rows * (stride + k) + 64,), float("nan"), dtype=dtype,
                         device="cuda")
        v = buf.as_strided((rows, C), (stride + k, 1), offset + k)
        if t is not None:
            v.copy_(t)
        return v, buf

    def around(v, buf):  # all NaN but the rows
        o = buf.clone()
        assert not v.isnan().any()
        o.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(float("nan"))
        return o.isnan().all()

    def weight(seed):
        return make((C + weights,), dtype, seed, 0.2, 1.0)[weights:]
    wp, g, wn = weight(3), weight(4), weight(5)
    x, a = make((rows, C), dtype, 1, 2.0), make((rows, C), dtype, 2, 0.5)
    w = dict(w_post=wp, gate=g, w_next=wn)
    (xv, _), (av, _), (yv, yb), (hv, hb) = lay(x), lay(a, 1), lay(None, 2), lay(None, 3)
    y, h, ra, ry = dash.join_fwd(xv, av, **w, eps=EPS, y=yv, h=hv)
    Y, H, RA, RY, ty, th = forward(x, a, wp, g, wn, 1.0, 1.0)
    near("y", y, Y, ty)
    near("h", h, H, th)
    assert around(yv, yb) and around(hv, hb)
    dy, dh = make((rows, C), dtype, 6), make((rows, C), dtype, 7)
    (dyv, _), (dhv, _), (dxv, dxb), (dav, dab) = lay(dy), lay(dh, 1), lay(None, 2), lay(None, 3)
    got = dash.join_bwd(dyv, dhv, yv, av, ra, ry, **w, dx=dxv, da=dav)
    want = backward(dy, dh, y, a, ra.double()[..., None], ry.double()[..., None], wp, g, wn, 1.0,
                    1.0)
    for n, t in zip(("dx", "da", "dw_post", "dgate", "dw_next"), got):
        near(n, t, *want[n])
    assert around(dxv, dxb) and around(dav, dab)
    # in place
    first, yv[:] = y.clone(), x
    dash.join_fwd(yv, av, **w, eps=EPS, y=yv, h=av)
    near("y in place", yv, Y, ty)
    near("h in place", av, H, th)
    if alike:
        assert torch.equal(yv, first) and torch.equal(av, h)


@pytest.mark.gpu
def test_join_gradient_against_differences(L):
    """<gradient, direction> against central differences of the definition in 64 bits, fp32
    rows.  The difference quotient is off by h^2 / 6 of the third derivative, at h = 1e-4 below
    1e-6 of the gradients' scale here; the gradients by 2^-16 of their terms."""
    shape, C = (2, 9, 200), 200
    t = dict(x=make(shape, F32, 1, 2.0), a=make(shape, F32, 2, 0.5),
             w_post=make((C,), F32, 3, 0.2, 1.0), gate=make((2, C), F32, 4, 0.5),
             w_next=make((C,), F32, 5, 0.2, 1.0))
    dy, dh = make(shape, F32, 6), make(shape, F32, 7)
    w = {k: t[k] for k in ("w_post", "gate", "w_next")}
    y, h, ra, ry = dash.join_fwd(t["x"], t["a"], **w, skip_scale=0.9, branch_scale=1.3, eps=EPS)
    got = dict(zip(("x", "a", "w_post", "gate", "w_next"),
                   dash.join_bwd(dy, dh, y, t["a"], ra, ry, **w, skip_scale=0.9, branch_scale=1.3)))

    def loss(d):
        Y, H, *_ = forward(d["x"], d["a"], d["w_post"], d["gate"], d["w_next"], 0.9, 1.3)
        return (Y * dy.double()).sum() + (H * dh.double()).sum()
    for n in t:
        g = torch.Generator(device="cuda").manual_seed(11)
        v = torch.randn(t[n].shape, generator=g, device="cuda", dtype=torch.float64)
        d = {k: u.double() for k, u in t.items()}
        hi = loss({**d, n: d[n] + 1e-4 * v})
        lo = loss({**d, n: d[n] - 1e-4 * v})
        want, have = (hi - lo) / 2e-4, (got[n].double() * v).sum()
        scale = (got[n].double() * v).abs().sum()
        assert abs(want - have) <= 2.0 ** -14 * scale, n


@pytest.mark.gpu
def test_rows_of_zeros_and_special_values(L):
    """A row of zeros stays finite (eps); a row with an infinity or NaN spoils its own rows and
    the weight gradients' columns only."""
    x, a = make((6, 256), BF, 1), make((6, 256), BF, 2)
    w = make((256,), BF, 3, 0.2, 1.0)
    x[1] = 0
    a[1] = 0
    x[3, 7] = float("inf")
    a[4, 9] = float("nan")
    y, h, ra, ry = dash.join_fwd(x, a, w_post=w, w_next=w)
    assert (y[1] == 0).all() and (h[1] == 0).all()
    for r in (0, 1, 2, 5):
        assert y[r].isfinite().all() and h[r].isfinite().all()
    assert y[3, 7].isinf() and y[4].isnan().all() and h[4].isnan().all()
    dx, da, *_ = dash.join_bwd(torch.ones_like(x), torch.ones_like(x), y, a, ra, ry, w_post=w,
                               w_next=w)
    for r in (0, 1, 2, 5):
        assert dx[r].isfinite().all() and da[r].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,pad", [(96, 8), (96, 3), (4096, 16), (17000, 8)])
def test_strides_in_place_and_bits(L, C, pad, dtype):
    """Rows at a stride (aligned and not), outputs that are inputs: the values of the contiguous
    call; the same bits on every run."""
    wide = make((40, 3 * (C + pad)), dtype, 1)
    x, a, dy = (wide[:, i * (C + pad): i * (C + pad) + C] for i in range(3))
    w = make((C,), dtype, 3, 0.2, 1.0)
    kw = dict(w_post=w, gate=w, w_next=w)
    y, h, ra, ry = dash.join_fwd(x.contiguous(), a.contiguous(), **kw)
    y2, h2, ra2, ry2 = dash.join_fwd(x, a, **kw)
    tight = dict(rtol=2.0 ** -7 if dtype == BF else 1e-5, atol=1e-5)
    for p, q in ((y, y2), (h, h2), (ra, ra2), (ry, ry2)):
        torch.testing.assert_close(p, q, **tight)
    first = dash.join_bwd(dy, h, y, a, ra, ry, **kw)
    for _ in range(3):
        again = dash.join_bwd(dy, h, y, a, ra, ry, **kw)
        assert all(torch.equal(p, q) for p, q in zip(first, again))
    keep = wide.clone()
    res = dash.join_fwd(x, a, **kw, y=x, h=a)
    assert res[0] is x and res[1] is a
    assert torch.equal(x, y2) and torch.equal(a, h2)
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[:, :C] = rest[:, C + pad: 2 * C + pad] = False
    assert torch.equal(wide[rest], keep[rest])


@pytest.mark.gpu
def test_stream_workspace_and_graph(L):
    x, a, dy = (make((300, 512), BF, i) for i in range(3))
    w = make((512,), BF, 3, 0.2, 1.0)
    kw = dict(w_post=w, w_next=w)
    y, h, ra, ry = dash.join_fwd(x, a, **kw)
    want = dash.join_bwd(dy, h, y, a, ra, ry, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dash.join_bwd(dy, h, y, a, ra, ry, **kw, stream=s)
    s.synchronize()
    assert all(g is None or torch.equal(g, v) for g, v in zip(got, want))
    ws = torch.empty(norms.join_bwd_workspace_bytes(300, 512, BF), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y2, h2, ra2, ry2 = dash.join_fwd(x, a, **kw)
        out = dash.join_bwd(dy, h2, y2, a, ra2, ry2, **kw, workspace=ws)
    g.replay()
    assert all(p is None or torch.equal(p, v) for p, v in zip(out, want))
    with pytest.raises(ValueError):
        dash.join_bwd(dy, h, y, a, ra, ry, **kw, workspace=ws[:100])


@pytest.mark.gpu
def test_refusals(L):
    x, w = torch.zeros(4, 6, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")

    def no(f, *a, **k):
        with pytest.raises(ValueError):
            f(*a, **k)
    no(dash.norm_fwd, x.cpu(), w)
    no(dash.norm_fwd, x.double(), w.double())
    no(dash.norm_fwd, x, w[:32])
    no(dash.norm_fwd, x, w.half())
    no(dash.norm_fwd, x, w.cpu())
    no(dash.norm_fwd, x, None)
    no(dash.norm_fwd, x.transpose(1, 2), w[:6])
    no(dash.norm_fwd, x[..., ::2], w[:32])
    no(dash.norm_fwd, x.transpose(0, 1), w)              # rows at no single stride
    no(dash.norm_fwd, x, w, out=x[:2])
    no(dash.norm_fwd, x, w, out=x.float())
    no(dash.norm_fwd, x, w, out=x[:1, :1].expand(4, 6, 64))
    no(dash.join_fwd, x, x[:2], w_next=w)
    no(dash.join_fwd, x, None, w_next=w)
    no(dash.join_fwd, x, x, w_post=w, w_next=w.float())  # weights of two types
    no(dash.join_fwd, x, x, gate=torch.ones(5, 64, dtype=BF, device="cuda"))
    no(dash.join_bwd, x, x, x, x, None, None, w_next=w)  # no rstd
    no(dash.join_bwd, None, None, x, x)
    rstd = torch.ones(4, 6, device="cuda")
    no(dash.join_bwd, x, x, x, x, None, rstd[:2], w_next=w)
    no(dash.norm_bwd, x, x, rstd.half(), w)
    no(dash.norm_bwd, x[:, :3], x, rstd, w)
    g = torch.ones(6, 64, dtype=BF, device="cuda")
    no(dash.join_fwd, x, x, gate=g)                      # torch would take a row for each token
    no(dash.join_fwd, x, x, gate=g[None])
    y = torch.zeros_like(x)
    no(dash.join_fwd, x, x, w_next=w, y=y, h=y)
    no(dash.join_bwd, x, x, x, x, None, rstd, w_next=w, dx=y, da=y)
    wide = torch.zeros(4, 6, 128, dtype=BF, device="cuda")
    no(dash.norm_fwd, wide[..., :64], w, out=wide.view(-1)[:1536].view(4, 6, 64))
    no(dash.norm_bwd, wide[..., :64], x, rstd, w, dx=wide.view(-1)[:1536].view(4, 6, 64))
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(8, device="cuda"),
               torch.zeros(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        no(dash.norm_bwd, x, x, rstd, w, workspace=ws)


def test_abi_refusals(L):
    fake, ll = 1 << 20, ctypes.c_longlong  # never dereferenced: every call is refused first

    def fwd(x=fake, a=fake, wp=fake, g=fake, wn=fake, y=fake, h=fake, ra=fake, ry=fake, rows=6, C=8,
            gr=3, dt=0, wdt=0, st=(ll * 4)(8, 8, 8, 8)):
        return L.dash_join_fwd(x, a, wp, g, wn, y, h, ra, ry, rows, C, gr, st, 1.0, 1.0, 1e-5, dt,
                               wdt, None)
    for bad in (dict(x=None), dict(y=None), dict(h=None), dict(ra=None), dict(ry=None),
                dict(rows=0), dict(C=0), dict(gr=4), dict(gr=0), dict(dt=3), dict(wdt=1),
                dict(dt=1, wdt=0), dict(x=fake + 1), dict(wp=fake + 1), dict(ra=fake + 2),
                dict(wdt=2, wn=fake + 2), dict(a=None), dict(st=None),
                dict(a=None, wp=None, g=None, wn=None)):
        assert fwd(**bad) == 1, bad
    assert fwd(rows=3 << 31) == 2 and fwd(C=1 << 25) == 2

    def bwd(dy=fake, dh=fake, y=fake, a=fake, wp=fake, g=fake, wn=fake, ra=fake, ry=fake, dx=fake,
            da=fake, dwp=fake, dg=fake, dwn=fake, ws=fake, n=1 << 30, rows=6, gr=3):
        return L.dash_join_bwd(dy, dh, y, a, wp, g, wn, ra, ry, dx, da, dwp, dg, dwn, rows, 8, gr,
                               (ll * 6)(*[8] * 6), 1.0, 1.0, 0, 0, ws, n, None)
    for bad in (dict(dx=None), dict(da=None), dict(dh=None), dict(y=None), dict(ry=None),
                dict(dwn=None), dict(ra=None), dict(dwp=None), dict(dg=None), dict(gr=4),
                dict(dy=fake + 1), dict(dwp=fake + 1), dict(dy=None, wn=None), dict(a=None)):
        assert bwd(**bad) == 1, bad
    assert bwd(ws=None) == 5 and bwd(n=8) == 5 and bwd(ws=fake + 8) == 5
    assert norms.norm_bwd_workspace_bytes(0, 8, BF) == 0
    assert norms.join_bwd_workspace_bytes(6, 8, BF, 4) == 0
    a = norms.join_bwd_workspace_bytes(6, 4096, BF)
    assert a >= 6 * 2 * 4096 * 4 and norms.norm_bwd_workspace_bytes(6, 4096, BF) < a


def test_abi_refuses_outputs_in_memory_that_is_read(L):
    """An output may be a row operand itself, not a weight, a gate, a row's rstd or another
    output: rows written early would be read as weights later."""
    ll = ctypes.c_longlong
    far = {n: (i + 1) << 24 for i, n in enumerate(  # never dereferenced: no device, or refused
        ("x", "a", "wp", "g", "wn", "y", "h", "ra", "ry"))}

    def fwd(**same):
        p = {**far, **{n: far[m] for n, m in same.items()}}
        return L.dash_join_fwd(*p.values(), 6, 8, 3, (ll * 4)(8, 8, 8, 8), 1.0, 1.0, 1e-5, 0, 0,
                               None)
    for out in ("y", "h"):
        for m in ("wp", "g", "wn"):
            assert fwd(**{out: m}) == 1, (out, m)
    assert fwd(y="h") == 1 and fwd(ra="ry") == 1 and fwd(ra="x") == 1 and fwd(ry="g") == 1
    far = {n: (i + 1) << 24 for i, n in enumerate(
        ("dy", "dh", "y", "a", "wp", "g", "wn", "ra", "ry", "dx", "da", "dwp", "dg", "dwn"))}

    def bwd(**same):
        p = {**far, **{n: far[m] for n, m in same.items()}}
        return L.dash_join_bwd(*p.values(), 6, 8, 1, (ll * 6)(*[8] * 6), 1.0, 1.0, 0, 0, 1 << 20,
                               1 << 30, None)
    for out in ("dx", "da", "dwp", "dg", "dwn"):
        for m in ("wp", "g", "wn", "ra", "ry"):
            assert bwd(**{out: m}) == 1, (out, m)
    assert bwd(dx="da") == 1 and bwd(dwp="dx") == 1 and bwd(dwn="dg") == 1


@pytest.mark.gpu
def test_refuses_outputs_that_are_weights(L):
    x = torch.ones(4, 6, 64, dtype=BF, device="cuda")
    one = torch.ones(1, 64, dtype=BF, device="cuda")
    w, rstd, gate = one[0], torch.ones(4, 6, device="cuda"), x.clone()

    def no(f, *a, **k):
        with pytest.raises(ValueError):
            f(*a, **k)
    no(dash.join_fwd, x, x, gate=gate, w_next=w, y=gate)
    no(dash.join_fwd, x, x, gate=gate, w_next=w, h=gate)
    no(dash.norm_fwd, one, w, out=one)                      # a row that is its weight
    for out in ("dx", "da"):
        no(dash.join_bwd, x, x, x, x, rstd, rstd, w_post=w, gate=gate, w_next=w, **{out: gate})
        no(dash.join_bwd, one, one, one, one, rstd[0, :1], rstd[0, :1], w_post=w, w_next=w.clone(),
           **{out: one})
    r = torch.ones(6, 1, device="cuda")                     # rows of one element in fp32
    no(dash.norm_bwd, r, r, r[:, 0], torch.ones(1, device="cuda"), dx=r)
    dash.join_bwd(x, x, x.clone(), x.clone(), rstd, rstd, w_post=w, gate=gate, w_next=w, dx=x)


@pytest.mark.gpu
def test_empty_batches_with_gates_and_outputs(L):
    """No sequences, or none of their tokens: a gate for every sequence goes with them, and so do
    outputs that the caller hands in (all at no address)."""
    w = make((64,), BF, 1)
    for shape, gate in (((0, 5, 64), (0, 64)), ((0, 5, 64), (0, 1, 64)), ((2, 0, 64), (2, 64)),
                        ((0, 64), (0, 64)), ((0, 5, 64), (0, 5, 64)), ((0, 5, 64), (64,))):
        x, g = torch.empty(shape, dtype=BF, device="cuda"), make(gate, BF, 2)
        kw = dict(w_post=w, gate=g, w_next=w)
        y, h, ra, ry = dash.join_fwd(x, x, **kw, y=torch.empty_like(x), h=torch.empty_like(x))
        assert y.shape == h.shape == x.shape and ra.shape == ry.shape == shape[:-1]
        dx, da, dwp, dg, dwn = dash.join_bwd(y, h, y, x, ra, ry, **kw, dx=torch.empty_like(x),
                                             da=torch.empty_like(x))
        assert dx.shape == da.shape == x.shape and dg.shape == g.shape
        assert (dwp == 0).all() and (dwn == 0).all() and (dg == 0).all()
    x = torch.empty(0, 5, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        dash.join_fwd(x, x, gate=make((0, 32), BF, 1))
    with pytest.raises(ValueError):
        dash.join_fwd(make((2, 5, 64), BF, 1), make((2, 5, 64), BF, 1), gate=make((0, 64), BF, 1))
