"""The operators on tensors of more than 2^31 elements: what lies furthest is right."""
import pytest
import torch

import deterministic_attention_backward_gb300 as dash

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def big(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=BF, device="cuda").normal_(generator=g)


@pytest.mark.parametrize("C", [4096, 4097])
def test_norm(C):
    """Last and first rows against 64 bits (fp32 sums of C terms: 2^-16 of theirs, a rounding of
    2^-8 each), the weight's gradient against its sum in 64 bits, 2^-16 of the terms' sum."""
    rows = 2 ** 31 // C + 1000
    x, dh, w = big(rows, C, seed=1), big(rows, C, seed=2), big(C, seed=3)
    h, rstd = dash.norm_fwd(x, w)
    dx, dw = dash.norm_bwd(dh, x, rstd, w)
    want, terms = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(2))
    for at in range(0, rows, 32768):
        part = slice(at, at + 32768)
        t = dh[part].double() * x[part].double() * rstd[part].double()[:, None]
        want += t.sum(0)
        terms += t.abs().sum(0)
    tol = 2.0 ** -16 * terms
    assert ((dw.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
    for part in (slice(0, 50), slice(rows - 50, rows)):
        X, D, W = x[part].double(), dh[part].double() * w.double(), w.double()
        r = (X.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
        H = X * r * W
        assert ((h[part].double() - H).abs() <= (2.0 ** -8 + 2.0 ** -15) * H.abs()).all()
        G = r * (D - X * r * (D * X * r).mean(-1, keepdim=True))
        t = r * (D.abs() + (X * r).abs() * (D * X * r).abs().mean(-1, keepdim=True))
        tol = 2.0 ** -15 * t
        assert ((dx[part].double() - G).abs() <= tol + 2.0 ** -8 * (G.abs() + tol)).all()


def test_rope():
    """The last tokens as the same tokens alone, turned from their own positions."""
    S, H, D = 2 ** 31 // (48 * 128) + 100, 48, 128
    q = big(1, S, H, D, seed=1)
    f, _ = dash.rope_freqs(D)
    want, _, _ = dash.rope_fwd(q[:, -200:], inv_freq=f, start=S - 200)
    got, _, _ = dash.rope_fwd(q, inv_freq=f)
    assert torch.equal(got[:, -200:], want)


def test_diff():
    """The last sequence as alone: O, O2, LSE and dQ bit for bit, dK and dV (whose key tiles may be
    cut otherwise) within their two roundings, 2^-8 each, and fp32 sums in another order."""
    B, S, H, Hkv, d = 65, 8192, 32, 8, 64
    q, k = big(B, S, 2 * H, d, seed=1), big(B, S, 2 * Hkv, d, seed=2)
    v, do = big(B, S, Hkv, 2 * d, seed=3), big(B, S, H, 2 * d, seed=4)
    lam = torch.linspace(0.1, 0.9, H, device="cuda")
    a = dash.diff_fwd(q, k, v, lam, causal=True, check=True)
    g = dash.diff_bwd(q, k, v, a[0], a[1], do, a[2], lam, causal=True, check=True)
    q, k, v, do = (t[-1:].clone() for t in (q, k, v, do))
    b = dash.diff_fwd(q, k, v, lam, causal=True)
    e = dash.diff_bwd(q, k, v, b[0], b[1], do, b[2], lam, causal=True)
    for x, y in zip((*a, g[0]), (*b, e[0])):
        assert torch.equal(x[-1:], y)
    for x, y in zip(g[1:3], e[1:3]):
        y = y.double()
        diff = (x[-1:].double() - y).abs()
        assert (diff <= 2 * 2.0 ** -8 * y.abs() + 2.0 ** -10 * y.abs().mean()).all()


def test_diff_weights_gradient():
    """dlam of more than 2^31 elements, summed from every sequence's tiles, against the sum of
    dO . O2 in 64 bits, O2 with what its rounding lost.  Values and dO are positive, so no terms
    cancel: a row's sum is off by P's rounding, 2^-8 / sqrt(3) of it in the root mean square, those
    of 532480 rows together by 2^-17, ten times less than the bound; one tile of the 4160 of a head
    that were left out or taken twice would be two times the bound."""
    B, S, H, Hkv, d = 65, 8192, 32, 8, 64
    q, k = big(B, S, 2 * H, d, seed=1), big(B, S, 2 * Hkv, d, seed=2)
    v, do = big(B, S, Hkv, 2 * d, seed=3).abs_(), big(B, S, H, 2 * d, seed=4).abs_()
    lam = torch.linspace(0.1, 0.9, H, device="cuda")
    rest = torch.empty(2, B, S, H, 2 * d, dtype=BF, device="cuda")
    o, o2, lse = dash.diff_fwd(q, k, v, lam, causal=True, check=True, rest=rest)
    *_, dlam = dash.diff_bwd(q, k, v, o, o2, do, lse, lam, causal=True, check=True, rest=rest)
    want = torch.zeros(H, dtype=torch.float64, device="cuda")
    for b in range(B):
        want -= (do[b].double() * (o2[b].double() + rest[1, b].double())).sum((0, 2))
    assert ((dlam.double() - want).abs() <= 2.0 ** -13 * want.abs()).all(), \
        (dlam.double() / want - 1).abs().max().item()
