"""Differential attention against its definition in 64 bits.

Tolerances, per element, from the roundings the kernels make.  bf16 rounds by at most half a
step, 2^-8 relative.  Scores are fp32 sums of products: off by at most 2^-20 of sum |q||k|
scale, which is below 50 here, so a probability is off by less than 2^-13 relative, with its
exp2 and the LSE's rounding less than r = 2^-12; sums of fp32 terms by 2^-16 of their absolute
values, also within r.
  forward    P is rounded:        t(Om) = (2^-8 + r) Pm |V|
  backward   P1 - lam P2 and dS are rounded, and carry r of their terms:
             t(P) = 2^-8 |P1 - lam P2| + 2 r (P1 + |lam| P2)
             t(dSm) = 2^-8 |dSm| + 2 r |lam_m| Pm (|dO||V|^T + sum |dO||Om|)
Each goes through its product with absolute values; the output's rounding adds 2^-8 (|x| + t)."""
import ctypes
import math

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build

BF, F32 = torch.bfloat16, torch.float32
HALF, R = 2.0 ** -8, 2.0 ** -12


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def make(B, S, H, Hkv, d, lam, seed=0, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    q = (spread * n(B, S, 2 * H, d)).to(BF)
    k, v, do = n(B, S, 2 * Hkv, d).to(BF), n(B, S, Hkv, 2 * d).to(BF), n(B, S, H, 2 * d).to(BF)
    kind, dtype = lam.split("-")
    w = n(*((H,) if kind == "head" else (B, S, H))) * 0.6 + 0.4  # some negative, some above 1
    return q, k, v, w.to({"bf16": BF, "fp32": F32}[dtype]), do


class Exact:
    """Everything in 64 bits, heads as [B, H, S, .]; P from the LSE that is given (the forward's
    own), D for dQ from the outputs that are given, for dK from P and dP, as the backward's
    contract has it."""

    def __init__(self, q, k, v, lam, causal, scale=None):
        B, S, H2, d = q.shape
        H, Hkv = H2 // 2, v.shape[2]
        G = H // Hkv
        self.dims = B, S, H, Hkv, G, d
        self.c = scale if scale else 1 / math.sqrt(d)
        self.q = q.double().view(B, S, H, 2, d).permute(3, 0, 2, 1, 4)
        self.k = k.double().view(B, S, Hkv, 2, d).permute(3, 0, 2, 1, 4).repeat_interleave(G, 2)
        self.v = v.double().transpose(1, 2).repeat_interleave(G, 1)
        s = self.q @ self.k.transpose(-1, -2) * self.c
        if causal:
            s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1), -math.inf)
        self.s = s
        self.lse = torch.logsumexp(s, -1)
        l = lam.double()
        self.lam = l[None, :, None, None] if l.dim() == 1 else l.transpose(1, 2)[..., None]
        self.per_head = l.dim() == 1

    def forward(self):
        P = (self.s - self.lse[..., None]).exp()
        o1, o2 = P[0] @ self.v, P[1] @ self.v
        t1, t2 = ((HALF + R) * (p @ self.v.abs()) for p in P)
        la = self.lam.abs()
        B, S, H, *_ = self.dims
        o, to, o2, t2 = (x.transpose(1, 2) for x in (o1 - self.lam * o2, t1 + la * t2, o2, t2))
        return {"o": (o, to), "o2": (o2, t2),
                "lse": (self.lse.permute(1, 2, 0, 3).reshape(B, 2 * H, S), None)}

    def backward(self, o, o2, do, lse):
        B, S, H, Hkv, G, d = self.dims
        o, o2, do = (t.double().transpose(1, 2) for t in (o, o2, do))
        lse = lse.double().view(B, H, 2, S).permute(2, 0, 1, 3)
        P = (self.s - lse[..., None]).exp()
        lam, la, c = self.lam, self.lam.abs(), self.c
        dP, dPa = do @ self.v.transpose(-1, -2), do.abs() @ self.v.abs().transpose(-1, -2)
        o1 = o + lam * o2
        D = torch.stack([(do * x).sum(-1, keepdim=True) for x in (o1, o2)])
        Da = torch.stack([(do.abs() * x).sum(-1, keepdim=True)
                          for x in (o.abs() + la * o2.abs(), o2.abs())])
        by = torch.stack([torch.ones_like(lam), -lam])
        dS = by * P * (dP - D)
        tS = HALF * dS.abs() + 2 * R * by.abs() * P * (dPa + Da)
        dSk = by * P * (dP - (P * dP).sum(-1, keepdim=True))
        tSk = HALF * dSk.abs() + 2 * R * by.abs() * P * (dPa + (P * dPa).sum(-1, keepdim=True))
        both = P[0] - lam * P[1]
        tP = HALF * both.abs() + 2 * R * (P[0] + la * P[1])

        def heads(t, n):  # [2, B, H, S, d] -> [B, S, 2n, d], the group's heads summed
            t = t.unflatten(2, (n, H // n)).sum(3)
            return t.permute(1, 3, 2, 0, 4).reshape(B, S, 2 * n, d)

        def values(t):
            return t.unflatten(1, (Hkv, G)).sum(2).transpose(1, 2)
        tr = (-1, -2)
        dl, tl = -(P[1] * dP).sum(-1), 2 * R * (P[1] * dPa).sum(-1)
        dl, tl = (x.sum((0, 2)) if self.per_head else x.transpose(1, 2) for x in (dl, tl))
        return {"dq": (heads(c * dS @ self.k, H), heads(c * tS @ self.k.abs(), H)),
                "dk": (heads(c * dSk.transpose(*tr) @ self.q, Hkv),
                       heads(c * tSk.transpose(*tr) @ self.q.abs(), Hkv)),
                "dv": (values(both.transpose(*tr) @ do), values(tP.transpose(*tr) @ do.abs())),
                "dlam": (dl, tl)}


def near(name, got, ref, tol):
    half = {BF: HALF, F32: 2.0 ** -24}[got.dtype]
    if name == "lse":
        tol = torch.full_like(ref, 2.0 ** -13)
    tol = tol + half * (ref.abs() + tol) + 1e-30
    err = (got.double() - ref).abs()
    assert got.shape == ref.shape
    assert (err <= tol).all(), f"{name}: over by {(err - tol).max().item():.3e}, " \
        f"largest share {(err / tol).max().item():.2f}"


def run(B, S, H, Hkv, d, causal, lam, seed=0, scale=None, spread=2.0):
    q, k, v, w, do = make(B, S, H, Hkv, d, lam, seed, spread)
    e = Exact(q, k, v, w, causal, scale)
    o, o2, lse = dash.diff_fwd(q, k, v, w, causal=causal, scale=scale, check=True)
    for n, g in (("o", o), ("o2", o2), ("lse", lse)):
        near(n, g, *e.forward()[n])
    grads = dash.diff_bwd(q, k, v, o, o2, do, lse, w, causal=causal, scale=scale, check=True)
    want = e.backward(o, o2, do, lse)
    for n, g in zip(("dq", "dk", "dv", "dlam"), grads):
        near(n, g, *want[n])
    return (q, k, v, w, do), (o, o2, lse), grads


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("S", [1, 2, 17, 63, 64, 65, 127, 128, 129, 192, 193, 256, 300, 515])
def test_lengths(L, S, causal, d):
    run(2, S, 2, 2, d, causal, "head-bf16", seed=S)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,S,H,Hkv", [(1, 200, 1, 1), (3, 130, 4, 2), (1, 390, 6, 1), (2, 77, 8, 8),
                                       (1, 1100, 3, 3)])
@pytest.mark.parametrize("lam", ["head-fp32", "token-bf16", "token-fp32"])
def test_heads_and_weights(L, lam, B, S, H, Hkv, causal, d):
    run(B, S, H, Hkv, d, causal, lam, seed=H + S)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,S,H,Hkv", [(1, 1300, 16, 16), (1, 2600, 1, 1), (1, 1500, 12, 3),
                                       (2, 900, 20, 20)])
def test_tiles_in_pieces(L, B, S, H, Hkv, causal, d):
    """Key tiles of which some or all are cut, into more pieces than the last ones have steps."""
    run(B, S, H, Hkv, d, causal, "head-bf16", seed=S)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
def test_scale_and_spread(L, causal, d):
    """A scale of one's own, flat and peaked maps: the running maximum stays and is raised."""
    run(1, 300, 2, 1, d, causal, "head-bf16", scale=0.07)
    run(1, 700, 2, 1, d, causal, "head-bf16", spread=0.01)
    run(1, 700, 2, 1, d, causal, "token-bf16", spread=5.0)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
def test_rising_scores(L, d):
    """Keys whose scores rise from block to block by far more than 2^8: every block rescales.
    Scores up to 600 scale the bound of their own rounding: 2^-20 x 1200, within 2^-9."""
    B, S, H = 1, 640, 1
    q, k, v, w, do = make(B, S, H, H, d, "head-bf16", 3)
    q = torch.ones_like(q)
    k = (torch.arange(S, device="cuda").view(1, S, 1, 1) // 128 * (15.0 / math.sqrt(d)) +
         0.1 * k.float()).to(BF)
    e = Exact(q, k, v, w, False)
    o, o2, lse = dash.diff_fwd(q, k, v, w, check=True)
    f = e.forward()
    near("o", o, f["o"][0], 2 * f["o"][1])
    near("o2", o2, f["o2"][0], 2 * f["o2"][1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
def test_gradient_against_differences(L, d):
    """<gradient, direction> against central differences of <O, dO> in 64 bits.  The gradient's
    own bounds, with what the rounded outputs add to D (their bounds times |dO|), weighted by the
    direction; the quotient's own error is far below (h^2 of third derivatives)."""
    for causal in (False, True):
        (q, k, v, w, do), (o, o2, lse), grads = run(1, 90, 2, 1, d, causal, "head-fp32", 5)
        e = Exact(q, k, v, w, causal)
        want = e.backward(o, o2, do, lse)
        f = e.forward()
        doa, la = do.double().abs().transpose(1, 2), e.lam.abs()
        t = [(doa * (x + HALF * y.abs()).transpose(1, 2)).sum(-1, keepdim=True)
             for y, x in (f["o"], f["o2"])]
        P = (e.s - e.lse[..., None]).exp()
        tS = torch.stack([P[0] * (t[0] + la * t[1]), la * P[1] * t[1]]) * e.c
        B, S, H, Hkv, G, _ = e.dims

        def heads(x, n):
            x = x.unflatten(2, (n, H // n)).sum(3)
            return x.permute(1, 3, 2, 0, 4).reshape(B, S, 2 * n, d)
        more = {"dq": heads(tS @ e.k.abs(), H), "dk": 0.0, "dv": 0.0, "dlam": 0.0}

        def loss(q, k, v, w):
            x = Exact(q, k, v, w, causal)
            P = (x.s - x.lse[..., None]).exp()
            return (((P[0] - x.lam * P[1]) @ x.v) * do.double().transpose(1, 2)).sum()
        for n, (x, name) in enumerate(zip((q, k, v, w), ("dq", "dk", "dv", "dlam"))):
            g = torch.Generator(device="cuda").manual_seed(n)
            u = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
            a = [t.double() for t in (q, k, v, w)]
            b = list(a)
            a[n], b[n] = a[n] + 1e-5 * u, b[n] - 1e-5 * u
            diff = (loss(*a) - loss(*b)) / 2e-5
            ref, tol = want[name]
            tol = tol + more[name] + HALF * (ref.abs() + tol)
            have = (grads[n].double() * u).sum()
            assert abs(have - diff) <= (tol * u.abs()).sum() + 1e-6 * abs(diff), (name, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64])
@pytest.mark.parametrize("causal", [False, True])
def test_equals_plain_attention_without_weight(L, d, causal):
    """lam = 0: the first map's plain attention of this library, at the head size both have."""
    q, k, v, w, do = make(1, 260, 2, 2, d, "head-fp32", 1)
    o, o2, _ = dash.diff_fwd(q, k, v, torch.zeros_like(w), causal=causal)
    for m, x in ((0, o), (1, o2)):
        for half in range(2):
            p, _ = dash.fwd(q[:, :, m::2].contiguous(), k[:, :, m::2].contiguous(),
                            v[..., half * d: half * d + d].contiguous(), causal=causal)
            a, b = x[..., half * d: half * d + d].double(), p.double()
            # both round P and the output: twice the forward's bound, |V| below 5
            assert ((a - b).abs() <= 4 * HALF * 5).all()
            assert (a - b).norm() <= 2 * HALF * b.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
def test_sequences_do_not_touch(L, d):
    """NaN and infinities in one sequence of a batch, at a length that ends inside a tile, leave
    the others' bits."""
    q, k, v, w, do = make(3, 100, 2, 1, d, "token-bf16", 2)
    o, o2, lse = dash.diff_fwd(q, k, v, w)
    g = dash.diff_bwd(q, k, v, o, o2, do, lse, w)
    for t, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, math.inf)):
        t[1] = bad
    p, p2, pl = dash.diff_fwd(q, k, v, w, check=True)
    h = dash.diff_bwd(q, k, v, p, p2, do, pl, w, check=True)
    for a, b in zip((o, o2, lse, *g), (p, p2, pl, *h)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    assert not p[1].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
def test_masked_keys_of_any_value(L, d):
    """Keys a causal row does not see may hold anything: NaN and infinities there leave the
    outputs of the rows before them as they were."""
    q, k, v, w, do = make(1, 200, 2, 2, d, "head-bf16", 2)
    o, o2, lse = dash.diff_fwd(q, k, v, w, causal=True)
    k[:, 150:] = math.nan
    k[:, 170:] = math.inf
    p, p2, pl = dash.diff_fwd(q, k, v, w, causal=True)
    for a, b in ((o, p), (o2, p2)):
        assert torch.equal(a[:, :150], b[:, :150])
    assert torch.equal(lse[..., :150], pl[..., :150])


@pytest.mark.gpu
@pytest.mark.parametrize("d,B,S,H,Hkv", [(64, 2, 700, 4, 2), (32, 3, 1237, 8, 8)])
@pytest.mark.parametrize("causal", [False, True])
def test_same_bits(L, d, B, S, H, Hkv, causal):
    q, k, v, w, do = make(B, S, H, Hkv, d, "head-bf16")
    first = None
    for n in range(4):
        o, o2, lse = dash.diff_fwd(q, k, v, w, causal=causal)
        got = (o, o2, lse, *dash.diff_bwd(q, k, v, o, o2, do, lse, w, causal=causal))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.gpu
def test_long_sequence(L):
    """A length whose tensors pass 2^31 bytes of scores per head; rows sampled."""
    B, S, H, Hkv, d = 1, 16500, 2, 1, 64
    q, k, v, w, do = make(B, S, H, Hkv, d, "head-bf16")
    o, o2, lse = dash.diff_fwd(q, k, v, w, causal=True, check=True)
    rows = torch.tensor([0, 127, 128, 8191, 16383, 16384, 16499], device="cuda")
    for h in range(H):
        s = torch.stack([q[0, rows, 2 * h + m].double() @ k[0, :, m].double().T / 8 for m in (0, 1)])
        s = s.masked_fill(torch.arange(S, device="cuda") > rows[:, None], -math.inf)
        P = s.softmax(-1)
        V = v[0, :, 0].double()
        lam = w[h].double()
        t = [(HALF + R) * (p @ V.abs()) for p in P]
        near("o", o[0, rows, h], (P[0] - lam * P[1]) @ V, t[0] + lam.abs() * t[1])
        near("o2", o2[0, rows, h], P[1] @ V, t[1])
        near("lse", lse[0, 2 * h: 2 * h + 2][:, rows], torch.logsumexp(s, -1), None)


@pytest.mark.gpu
def test_stream_workspace_and_graph(L):
    q, k, v, w, do = make(1, 300, 4, 2, 64, "head-bf16")
    o, o2, lse = dash.diff_fwd(q, k, v, w, causal=True)
    want = dash.diff_bwd(q, k, v, o, o2, do, lse, w, causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = dash.diff_fwd(q, k, v, w, causal=True, stream=s)
    got = dash.diff_bwd(q, k, v, a[0], a[1], do, a[2], w, causal=True, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    n = dash.diff_bwd_workspace_bytes(1, 300, 4, 64)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")  # need not be initialised
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x = dash.diff_fwd(q, k, v, w, causal=True, workspace=ws)
        got = dash.diff_bwd(q, k, v, x[0], x[1], do, x[2], w, causal=True, workspace=ws)
    q2, k2, v2, w2, do2 = make(1, 300, 4, 2, 64, "head-bf16", 9)
    o, o2, lse = dash.diff_fwd(q2, k2, v2, w2, causal=True)
    want = dash.diff_bwd(q2, k2, v2, o, o2, do2, lse, w2, causal=True)
    for t, u in ((q, q2), (k, k2), (v, v2), (w, w2), (do, do2)):
        t.copy_(u)
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    dash.status(ws)
    with pytest.raises(ValueError):
        dash.diff_bwd(q, k, v, o, o2, do, lse, w, workspace=ws[:-256])


@pytest.mark.gpu
def test_nothing_to_do(L):
    for B, S in ((0, 5), (2, 0)):
        q, k, v, w, do = make(B, S, 2, 1, 64, "head-bf16")
        o, o2, lse = dash.diff_fwd(q, k, v, w)
        dq, dk, dv, dlam = dash.diff_bwd(q, k, v, o, o2, do, lse, w)
        assert o.shape == (B, S, 2, 128) and lse.shape == (B, 4, S) and dk.shape == k.shape
        assert (dlam == 0).all() and dlam.shape == w.shape


@pytest.mark.gpu
def test_refusals(L):
    q, k, v, w, do = make(1, 8, 4, 2, 64, "head-bf16")

    def no(*a, **kw):
        with pytest.raises(ValueError):
            dash.diff_fwd(*a, **kw)
    no(q.float(), k, v, w)
    no(q.cpu(), k, v, w)
    no(q[:, :, :7], k, v, w)                      # not contiguous, and no pairs
    no(q[:, :, :7].contiguous(), k, v, w)
    no(q[:, :, :6].contiguous(), k, v, w[:3])     # no whole group
    no(q, k[:, :4].contiguous(), v, w)
    no(q, k, v[..., :64].contiguous(), w)
    no(q, k, v, w[:3])
    no(q, k, v, w.half())
    no(q, k, v, w.cpu())
    no(q[0], k, v, w)
    no(q.transpose(1, 2), k, v, w)
    no(q, k, v, w, out=do[:, :4])
    no(q, k, v, w, out2=do.float())
    o, o2, lse = dash.diff_fwd(q, k, v, w)
    for bad in (dict(o=o[:, :4]), dict(lse=lse.double()), dict(lse=lse[:, :4]), dict(do=do.float())):
        a = dict(o=o, o2=o2, do=do, lse=lse, **{})
        a.update(bad)
        with pytest.raises(ValueError):
            dash.diff_bwd(q, k, v, a["o"], a["o2"], a["do"], a["lse"], w)
    no(q, k, v, w, out=o, out2=o)
    host = torch.zeros(1 << 20, dtype=torch.uint8)
    no(q, k, v, w, workspace=host)
    no(q, k, v, w, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    for bad in (dict(dq=q), dict(dk=k), dict(dlam=w), dict(workspace=host)):
        with pytest.raises(ValueError):
            dash.diff_bwd(q, k, v, o, o2, do, lse, w, **bad)
    x, y, z, u, _ = make(1, 8, 2, 2, 16, "head-bf16")
    with pytest.raises(dash.DashError) as err:
        dash.diff_fwd(x, y, z, u)
    assert err.value.code == 2


def test_abi_refusals(L):
    fake = 1 << 20  # never dereferenced: every call is refused first

    def fwd(ptrs=None, lam=fake, lse=fake, B=1, S=8, H=4, G=2, d=64, mask=0, ldt=0, ws=fake, n=256):
        p = ptrs or [fake] * 5
        return L.dash_diff_fwd(p[0], p[1], p[2], lam, p[3], p[4], lse, B, S, H, G, d, 0.0, mask, ldt,
                               0, ws, n, None)
    for bad in (dict(B=0), dict(S=0), dict(H=0), dict(G=3), dict(d=0), dict(mask=2), dict(ldt=1),
                dict(lam=None), dict(lam=fake + 1), dict(lam=fake + 2, ldt=2), dict(lse=None),
                dict(lse=fake + 2), dict(ptrs=[fake, fake, None, fake, fake]),
                dict(ptrs=[fake, fake, fake, fake, fake + 8])):
        assert fwd(**bad) == 1, bad
    assert fwd(d=128) == 2 and fwd(B=1 << 16, S=1 << 15) == 2
    assert fwd(ws=None) == 5 and fwd(n=255) == 5 and fwd(ws=fake + 8) == 5

    def bwd(ptrs=None, lam=fake, dlam=fake, lse=fake, S=8, ws=fake, n=1 << 30):
        p = ptrs or [fake] * 9
        return L.dash_diff_bwd(*p[:6], lse, lam, *p[6:], dlam, 1, S, 4, 2, 64, 0.0, 1, 0, 0, ws, n,
                               None)
    for bad in (dict(S=0), dict(lam=None), dict(dlam=None), dict(lse=None),
                dict(ptrs=[fake] * 8 + [None]), dict(ptrs=[fake + 8] + [fake] * 8)):
        assert bwd(**bad) == 1, bad
    n = dash.diff_bwd_workspace_bytes(1, 8, 4, 64)
    assert bwd(ws=None) == 5 and bwd(n=n - 1) == 5
    assert n >= 256 + 4 * 128 * 20 and dash.diff_bwd_workspace_bytes(1, 8, 4, 96) == 0
    assert L.dash_diff_fwd_workspace_bytes(1, 8, 4, 32) == 256


def with_rest(q, k, v, w, do, causal, **kw):
    rest = torch.full((2, *do.shape), math.nan, dtype=BF, device="cuda")
    o, o2, lse = dash.diff_fwd(q, k, v, w, causal=causal, check=True, rest=rest, **kw)
    return (o, o2, lse, rest), dash.diff_bwd(q, k, v, o, o2, do, lse, w, causal=causal, check=True,
                                             rest=rest, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("S,H,Hkv,lam", [(1, 1, 1, "head-bf16"), (17, 2, 1, "token-fp32"),
                                         (129, 4, 2, "head-fp32"), (300, 2, 2, "token-bf16"),
                                         (1030, 3, 1, "head-bf16")])
def test_rest_of_the_outputs(L, S, H, Hkv, lam, causal, d):
    """rest adds what O and O2 lose: the sum is off by what P's rounding gives, (2^-8 + r) of the
    terms, and twice a rounding, 2^-16 of the value.  All else is what the calls give without it,
    bit for bit, but dQ."""
    q, k, v, w, do = make(2, S, H, Hkv, d, lam, seed=S)
    (o, o2, lse, rest), grads = with_rest(q, k, v, w, do, causal)
    f = Exact(q, k, v, w, causal).forward()
    for n, x, y in (("o", o, rest[0]), ("o2", o2, rest[1])):
        ref, tol = f[n]
        both = x.double() + y.double()
        assert (y.double().abs() <= HALF * x.double().abs() * (1 + HALF)).all()
        assert ((both - ref).abs() <= tol * (1 + 2 * HALF) + 2.0 ** -16 * ref.abs()).all()
    p = dash.diff_fwd(q, k, v, w, causal=causal)
    assert all(torch.equal(a, b) for a, b in zip((o, o2, lse), p))
    plain = dash.diff_bwd(q, k, v, o, o2, do, lse, w, causal=causal)
    assert all(torch.equal(a, b) for a, b in zip(grads[1:], plain[1:]))
    zero = dash.diff_bwd(q, k, v, o, o2, do, lse, w, causal=causal, rest=torch.zeros_like(rest))
    assert all(torch.equal(a, b) for a, b in zip(zero, plain))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("spread", [1.0, 2.0, 4.0, 8.0])
def test_dq_with_rest(L, spread, causal, d):
    """dQ against its definition in 64 bits, D from P and dP, in the Euclidean norm.  Roundings are
    off by 2^-8 of the value at most, evenly spread, 2^-8 / sqrt(3) in the root mean square, each
    its own way.  Three reach dQ: its own; dS's, through dS K; P's in the forward, through
    D = sum P dP and P K.  Their squares add up (two more of D's, 2^-16, and r do not count)."""
    S, H = 700, 2
    q, k, v, w, do = make(1, S, H, H, d, "head-fp32", seed=7, spread=spread)
    w = torch.tensor([0.8, 1.0], device="cuda")
    _, (dq, *_) = with_rest(q, k, v, w, do, causal)
    e = Exact(q, k, v, w, causal)
    P = (e.s - e.lse[..., None]).exp()
    dP = do.double().transpose(1, 2) @ e.v.transpose(-1, -2)
    by = torch.stack([torch.ones_like(e.lam), -e.lam])
    dS = by * P * (dP - (P * dP).sum(-1, keepdim=True))
    offD = (P * dP).square().sum(-1, keepdim=True)
    for m in range(2):
        want = e.c * dS[m] @ e.k[m]
        got = dq.double().view(1, S, H, 2, d)[:, :, :, m].transpose(1, 2)
        inner = e.c ** 2 * (dS[m].square() @ e.k[m].square() +
                            by[m].square() * offD[m] * (P[m] @ e.k[m]).square())
        tol = HALF / 3 ** 0.5 * (want.square().sum() + inner.sum()).sqrt()
        assert (got - want).norm() <= tol, ((got - want).norm() / want.norm()).item()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
def test_dq_of_a_row_that_sees_one_key(L, d):
    """dQ is zero: P = 1, and D = dO . V1 comes back from O + lam O2 with two roundings of 2^-16 of
    the terms (2^-15 with the fp32 sums), times one key."""
    q, k, v, w, do = make(3, 200, 4, 2, d, "token-fp32", seed=2, spread=4.0)
    (o, o2, *_), (dq, *_) = with_rest(q, k, v, w, do, True)
    a = do[:, 0].double().abs()
    own = v[:, 0].double().abs().repeat_interleave(2, 1)
    lam = w[:, 0].double().abs()[..., None]
    terms = (a * (o[:, 0].double().abs() + lam * o2[:, 0].double().abs() + own)).sum(-1)
    key = k[:, 0].double().abs().view(3, 2, 2, d).repeat_interleave(2, 1)  # [B, H, 2, d]
    tol = 2.0 ** -15 * terms[..., None, None] * key / math.sqrt(d)
    tol[:, :, 1] *= lam
    assert (dq[:, 0].double().abs().view(3, 4, 2, d) <= tol * (1 + HALF)).all()


@pytest.mark.gpu
def test_rest_refusals(L):
    q, k, v, w, do = make(1, 8, 4, 2, 64, "head-bf16")
    o, o2, lse = dash.diff_fwd(q, k, v, w)
    rest = torch.empty(2, *do.shape, dtype=BF, device="cuda")
    both = torch.empty(3, *do.shape, dtype=BF, device="cuda")
    for bad in (rest[0], rest[:1], rest.float(), rest.cpu(), rest.transpose(0, 1)):
        with pytest.raises(ValueError):
            dash.diff_fwd(q, k, v, w, rest=bad)
        with pytest.raises(ValueError):
            dash.diff_bwd(q, k, v, o, o2, do, lse, w, rest=bad)
    for kw in (dict(out=rest[0], rest=rest), dict(out2=both[1], rest=both[:2])):
        with pytest.raises((ValueError, dash.DashError)):
            dash.diff_fwd(q, k, v, w, **kw)
    with pytest.raises((ValueError, dash.DashError)):
        dash.diff_bwd(q, k, v, o, o2, do, lse, w, rest=both[:2], dv=both.view(-1)[:v.numel()].view(
            v.shape))
    for B, S in ((0, 5), (2, 0)):
        x, y, z, u, g = make(B, S, 2, 1, 64, "head-bf16")
        out, grads = with_rest(x, y, z, u, g, True)
        assert out[0].shape == g.shape and (grads[3] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(64, True), (64, False), (32, True)])
def test_long_sequence_backward(L, d, causal):
    """64 key blocks and query tiles: every gradient against 64 bits.  dK sums 16384 queries in
    1024 additions of 16, which is within 2^-14 of the terms, so within r as before."""
    run(1, 8192, 2, 1, d, causal, "head-bf16", seed=4)
    torch.cuda.empty_cache()


def test_forward_workspace_bytes(L):
    """The size that a caller's own workspace of the forward needs, and no size where it has none."""
    n = dash.diff_fwd_workspace_bytes(2, 300, 4, 64)
    assert n == L.dash_diff_fwd_workspace_bytes(2, 300, 4, 64) == 256
    assert dash.diff_fwd_workspace_bytes(2, 300, 4, 96) == 0
    assert "diff_fwd_workspace_bytes" in dash.__all__


@pytest.mark.gpu
def test_rest_on_another_stream_and_captured(L):
    q, k, v, w, do = make(2, 333, 4, 2, 64, "head-bf16")
    (o, o2, lse, rest), want = with_rest(q, k, v, w, do, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(rest)
    a = dash.diff_fwd(q, k, v, w, causal=True, stream=s, rest=other)
    got = dash.diff_bwd(q, k, v, a[0], a[1], do, a[2], w, causal=True, stream=s, rest=other)
    s.synchronize()
    assert torch.equal(other, rest) and all(torch.equal(x, y) for x, y in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x = dash.diff_fwd(q, k, v, w, causal=True, rest=other)
        got = dash.diff_bwd(q, k, v, x[0], x[1], do, x[2], w, causal=True, rest=other)
    new = make(2, 333, 4, 2, 64, "head-bf16", 9)
    (_, _, _, rest), want = with_rest(*new, True)
    for t, u in zip((q, k, v, w, do), new):
        t.copy_(u)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, rest) and all(torch.equal(x, y) for x, y in zip(got, want))
