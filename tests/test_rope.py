"""Rotary positions against the definition in 64 bits.

Tolerance.  The kernel's angle is off by at most 2^-25 half turns (the fp32 rounding of the
phase) and sincospif by two units in the last place, so cos and sin are off by less than
pi 2^-25 + 2^-22 < 2^-21; the turn of a pair of norm n then by 2 n 2^-21 with its own fp32
rounding (three roundings of 2^-24 relative to n) below that: 2^-19 n m in all for magnitude m.
Rounding to the output's type adds half a step, eps / 2 relative to the value."""
import math

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build
from deterministic_attention_backward_gb300.rope import _PART

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def reference(x, inv_freq, m, pos, layout, back):
    """x [B,S,H,D] float64, pos [B,S] int64: the turned heads and each element's pair norm."""
    n = inv_freq.numel()
    # float64 angles: off by 2^-53 of the angle, 2^-22 radians at position 2^31
    a = pos.double()[:, :, None, None] * inv_freq.double()
    c, s = a.cos() * m, a.sin() * (-m if back else m)
    i = torch.arange(n)
    lo, hi = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    lo, hi = lo.to(x.device), hi.to(x.device)
    out, norm = x.clone(), torch.zeros_like(x)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    r = (x[..., lo] ** 2 + x[..., hi] ** 2).sqrt()
    norm[..., lo] = r
    norm[..., hi] = r
    return out, norm


def check(got, x, inv_freq, m, pos, layout, back):
    ref, norm = reference(x.double(), inv_freq, m, pos, layout, back)
    tol = 2.0 ** -19 * m * norm
    if got.dtype != F32:
        tol = tol + torch.finfo(got.dtype).eps / 2 * (ref.abs() + tol)
        tol = tol + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (err - tol).max().item()


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def test_frequencies():
    f, m = dash.rope_freqs(8, base=10000.0, device="cpu")
    assert m == 1.0 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001]).double(), rtol=1e-6)
    f4, _ = dash.rope_freqs(8, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(f4, f / 4)
    fb, _ = dash.rope_freqs(8, scaling="base", factor=4.0, device="cpu")
    assert math.isclose(fb[-1], f[-1] / 4, rel_tol=1e-12) and fb[0] == f[0]
    f, _ = dash.rope_freqs(128, device="cpu")
    fr, m = dash.rope_freqs(128, scaling="ramp", factor=16.0, original_len=4096, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(fr[turns > 32], f[turns > 32])
    assert torch.allclose(fr[turns < 1], f[turns < 1] / 16, rtol=1e-12)
    assert (fr[:-1] > fr[1:]).all() and math.isclose(m, 0.1 * math.log(16) + 1)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, scaling="other"), dict(rot=8, factor=0.0),
                dict(rot=8, scaling="ramp", fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            dash.rope_freqs(device="cpu", **bad)


def test_abi_refusals(L):
    fake = 1 << 20  # never dereferenced: every call below is refused first

    def call(nparts=1, B=1, S=1, rot=8, layout=0, dtype=0, freq=fake, pos=None, pos64=0, **part):
        q = {**dict(inp=fake, out=fake, heads=2, D=16, turn=1), **part}
        a = _PART.pack(q["inp"] or 0, q["out"] or 0, q["heads"], q["D"], q["turn"], *[16] * 6) * 4
        return L.dash_rope(a, nparts, B, S, rot, layout, dtype, freq, 1.0, pos, pos64, 0, 1, 0, 0,
                           None)
    for bad in (dict(nparts=0), dict(nparts=4), dict(B=0), dict(S=-1), dict(rot=7), dict(rot=0),
                dict(rot=18), dict(layout=2), dict(dtype=3), dict(freq=None), dict(freq=fake + 4),
                dict(pos=fake + 2), dict(pos=fake + 4, pos64=1), dict(inp=None), dict(out=None),
                dict(inp=fake + 1), dict(heads=0), dict(D=0)):
        assert call(**bad) == 1, bad
    assert call(rot=1026, D=2048) == 2
    assert call(B=1 << 20, S=1 << 12) == 2
    assert L.dash_rope(None, 1, 1, 1, 8, 0, 0, fake, 1.0, None, 0, 0, 1, 0, 0, None) == 1


CASES = [  # B, S, H, Hkv, D, rot, layout
    (1, 1, 1, 1, 2, 2, "half"),
    (2, 3, 4, 2, 64, 64, "half"),
    (1, 5, 3, 1, 96, 48, "interleaved"),
    (2, 7, 2, 2, 20, 10, "half"),           # single elements
    (2, 7, 2, 2, 20, 10, "interleaved"),
    (1, 33, 5, 5, 128, 32, "half"),
    (3, 1237, 4, 2, 64, 64, "interleaved"),  # several tokens to a CTA, a partial last one
    (1, 2500, 3, 1, 72, 24, "half"),
    (1, 2, 1, 1, 1024, 1024, "half"),
]


def make(B, S, h, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, S, h, D, generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_matches_definition(L, case, dtype, back):
    B, S, H, Hkv, D, rot, layout = case
    f, m = dash.rope_freqs(rot, scaling="ramp", factor=4.0)
    q, k, v = (make(B, S, h, D, dtype, i) for i, h in enumerate((H, Hkv, Hkv)))
    pos = torch.arange(S, device="cuda").expand(B, S) + 1000003
    fn = dash.rope_bwd if back else dash.rope_fwd
    got = fn(q, k, v, inv_freq=f, magnitude=m, start=1000003, layout=layout)
    check(got[0], q, f, m, pos, layout, back)
    check(got[1], k, f, m, pos, layout, back)
    assert torch.equal(got[2], v) and got[2].data_ptr() != v.data_ptr()
    assert all(t.is_contiguous() for t in got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_positions(L, dtype):
    """Given positions in any order, negative and beyond 32 bits of phase; per batch and shared;
    strided; packed heads."""
    f, _ = dash.rope_freqs(64)
    q = make(2, 6, 3, 64, F32, 0)
    pos = torch.tensor([[5, 5, 0, -7, 2 ** 31 - 1, 123456789], [0, 1, 2, 3, 4, -2 ** 31]],
                       device="cuda").to(dtype)
    got = dash.rope_fwd(q, inv_freq=f, positions=pos)
    assert got[1] is None and got[2] is None
    check(got[0], q, f, 1.0, pos.long(), "half", False)
    check(dash.rope_fwd(q, inv_freq=f, positions=pos[0])[0], q, f, 1.0,
          pos[:1].long().expand(2, 6), "half", False)
    wide = torch.zeros(2, 12, dtype=dtype, device="cuda")
    wide[:, ::2] = pos
    assert torch.equal(dash.rope_fwd(q, inv_freq=f, positions=wide[:, ::2])[0], got[0])
    packed = dash.rope_fwd(q.view(12, 3, 64), inv_freq=f, positions=pos.reshape(12))[0]
    assert torch.equal(packed.view(2, 6, 3, 64), got[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("offset", [0, 1])
def test_strided_views_and_in_place(L, dtype, offset):
    """Views of one qkv product (and of one whose heads start off a 16-byte boundary) in, views
    of its gradient out, in place: the bits of the contiguous call."""
    B, S, H, Hkv, D = 2, 37, 4, 2, 64
    f, _ = dash.rope_freqs(D)
    qkv = make(B, S, 1, (H + 2 * Hkv) * D + 8, dtype, 3)[:, :, 0]
    parts = [t.unflatten(-1, (-1, D)) for t in
             qkv[..., offset: offset + (H + 2 * Hkv) * D].split([H * D, Hkv * D, Hkv * D], dim=-1)]
    want = dash.rope_fwd(*[t.contiguous() for t in parts], inv_freq=f)
    got = dash.rope_fwd(*parts, inv_freq=f)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out = torch.full_like(qkv, 7.0)
    views = tuple(t.unflatten(-1, (-1, D)) for t in
                  out[..., offset: offset + (H + 2 * Hkv) * D].split([H * D, Hkv * D, Hkv * D],
                                                                     dim=-1))
    res = dash.rope_fwd(*parts, inv_freq=f, out=views)
    assert all(r is v for r, v in zip(res, views))
    assert all(torch.equal(a, b) for a, b in zip(want, views))
    assert (out[..., :offset] == 7).all() and (out[..., offset + (H + 2 * Hkv) * D:] == 7).all()
    q = want[0].clone()
    dash.rope_bwd(q, inv_freq=f, out=(q, None, None))  # in place: turned back
    n = torch.finfo(dtype).eps if dtype == BF else 2.0 ** -18
    r = parts[0].double()
    pair = (r.view(B, S, H, 2, D // 2) ** 2).sum(-2).sqrt().repeat(1, 1, 1, 2)
    assert ((q.double() - r).abs() <= 2 * n * pair).all()


@pytest.mark.gpu
def test_backward_is_the_gradient(L):
    """<dq, rope(u)> = <rope_bwd(dq), u> for random u: the transpose, magnitude included."""
    f, m = dash.rope_freqs(48, scaling="ramp", factor=8.0)
    u, dq = make(1, 50, 3, 96, F32, 1), make(1, 50, 3, 96, F32, 2)
    a = (dq.double() * dash.rope_fwd(u, inv_freq=f, magnitude=m, start=9)[0].double()).sum()
    b = (u.double() * dash.rope_bwd(dq, inv_freq=f, magnitude=m, start=9)[0].double()).sum()
    # each of the n products is off by 2^-19 m |u||dq|: below 2^-19 m ||u|| ||dq||
    assert abs(a - b) <= 2 * 2.0 ** -19 * m * u.double().norm() * dq.double().norm()


@pytest.mark.gpu
def test_nothing_to_do_and_special_values(L):
    f, _ = dash.rope_freqs(64)
    for shape in ((0, 4, 2, 64), (2, 0, 2, 64), (2, 4, 0, 64)):
        assert dash.rope_fwd(torch.zeros(shape, dtype=BF, device="cuda"), inv_freq=f)[0].shape == shape
    x = make(1, 4, 2, 64, BF, 0)
    x[0, 1, 0, 3] = math.inf
    x[0, 2, 1, 40] = math.nan
    y = dash.rope_fwd(x, inv_freq=f, start=1)[0]
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[0, 1, 0, [3, 35]] = True
    bad[0, 2, 1, [8, 40]] = True
    assert torch.equal(~y.isfinite(), bad)


@pytest.mark.gpu
def test_stream_and_graph(L):
    f, _ = dash.rope_freqs(64)
    x = make(1, 300, 4, 64, BF, 0)
    want = dash.rope_fwd(x, inv_freq=f)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dash.rope_fwd(x, inv_freq=f, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dash.rope_fwd(x, inv_freq=f, out=(out, None, None))
    y = make(1, 300, 4, 64, BF, 5)
    x.copy_(y)
    g.replay()
    assert torch.equal(out, dash.rope_fwd(y, inv_freq=f)[0])


@pytest.mark.gpu
def test_refusals(L):
    f, _ = dash.rope_freqs(64)
    q = torch.zeros(2, 4, 2, 64, dtype=BF, device="cuda")

    def no(*a, **k):
        with pytest.raises(ValueError):
            dash.rope_fwd(*a, **{**dict(inv_freq=f), **k})
    no(q.cpu())
    no(q.double())
    no(q[0, 0])
    no(q.transpose(2, 3))
    no(q[..., :32])                                      # fewer elements than turn
    no(q, q[:, :3])
    no(q, q.float())
    no(q, inv_freq=f.float())
    no(q, inv_freq=f.cpu())
    no(q, inv_freq=f[::2])
    no(q, layout="other")
    no(q, positions=torch.zeros(3, dtype=torch.int64, device="cuda"))
    no(q, positions=torch.zeros(4, device="cuda"))
    no(q, positions=torch.zeros(4, dtype=torch.int64))
    no(q, out=(q,))
    no(q, out=(q[:, :3], None, None))
    no(q, out=(q[:1].expand(2, 4, 2, 64), None, None))   # shared addresses
    k, o = torch.zeros_like(q), torch.zeros_like(q)
    no(q, k, out=(o, o, None))
    no(q, k, out=(k, o, None))
    no(q, k, out=(o, q, None))
    wide = torch.zeros(2, 8, 2, 64, dtype=BF, device="cuda")
    no(wide[:, :4], out=(wide.view(-1)[:1024].view(2, 4, 2, 64), None, None))  # other strides


def turns(inv_freq, pos):
    """pos inv_freq / (2 pi) modulo 1, exact up to 2^-200: pi by Machin's formula in integers."""
    from fractions import Fraction

    def arctan(n, bits=400):  # of 1 / n
        term = total = (1 << bits) // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total
    two_pi = Fraction(8 * (4 * arctan(5) - arctan(239)), 1 << 400)
    return float(Fraction(inv_freq) * pos / two_pi % 1)


@pytest.mark.gpu
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_positions(L, base):
    """Positions over all of 64 bits.  The pair (1, 0) becomes (cos a, sin a), each off by less than
    2^-21 as above: nothing of the angle is lost on the way to its last fp32 rounding."""
    f, _ = dash.rope_freqs(128, base=base)
    far = [2 ** 31 - 1, 2 ** 36 + 5, 2 ** 40 - 3, 2 ** 53 + 1, 2 ** 62 + 12345, 2 ** 63 - 1, -2 ** 63,
           -2 ** 45 - 1, 0]
    pos = torch.tensor([far], device="cuda")
    x = torch.zeros(1, len(far), 1, 128, device="cuda")
    x[..., :64] = 1.0
    got = dash.rope_fwd(x, inv_freq=f, positions=pos)[0][0, :, 0].double().cpu()
    for row, p in zip(got, far):
        a = torch.tensor([2 * math.pi * turns(w, p) for w in f.tolist()], dtype=torch.float64)
        err = (row - torch.cat([a.cos(), a.sin()])).abs().max().item()
        assert err < 2.0 ** -21, (p, err)
        alone = dash.rope_fwd(x[:, :1], inv_freq=f, start=p)[0][0, 0, 0].double().cpu()
        assert torch.equal(alone, row)


@pytest.mark.gpu
def test_frequencies_that_are_no_numbers(L):
    """A frequency that is infinite or NaN has no angle: its pair is NaN, the others are turned."""
    f, _ = dash.rope_freqs(64)
    x = make(1, 3, 2, 64, BF, 0)
    want = dash.rope_fwd(x, inv_freq=f, start=5)[0]
    for p, bad in ((0, math.nan), (7, math.inf), (31, -math.inf)):
        g = f.clone()
        g[p] = bad
        for start in (5, 0):
            y = dash.rope_fwd(x, inv_freq=g, start=start)[0]
            assert y[..., [p, p + 32]].isnan().all()
            keep = [i for i in range(64) if i not in (p, p + 32)]
            assert start == 0 or torch.equal(y[..., keep], want[..., keep])


@pytest.mark.gpu
def test_start_beyond_64_bits(L):
    f, _ = dash.rope_freqs(64)
    x = make(1, 3, 2, 64, BF, 0)
    for start in (2 ** 63, -2 ** 63 - 1, 2 ** 70, 2 ** 63 - 2):
        with pytest.raises(ValueError):
            dash.rope_fwd(x, inv_freq=f, start=start)
    dash.rope_fwd(x, inv_freq=f, start=2 ** 63 - 3)
    dash.rope_fwd(x, inv_freq=f, positions=torch.zeros(3, dtype=torch.int64, device="cuda"))


def test_ramp_is_the_published_one():
    """Frequencies for longer contexts by parts (YaRN, arXiv 2309.00071, with its ramp over the pair
    index): a pair n turns around L / (2 pi) base^(-2n/rot) times, the ramp runs from the floor of
    the index at which that is `fast` to the ceiling of that at which it is `slow`."""
    for rot, base, L, factor in ((128, 1e4, 4096, 4.0), (128, 1e4, 4096, 32.0), (64, 5e5, 8192, 8.0),
                                 (32, 1e4, 131072, 2.0), (128, 1e4, 4096, 1.0), (8, 1e6, 100, 4.0)):
        fr, m = dash.rope_freqs(rot, base=base, scaling="ramp", factor=factor, original_len=L,
                                device="cpu")

        def index(turns):
            return rot * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(index(32)), 0), min(math.ceil(index(1)), rot - 1)
        for n, got in enumerate(fr.tolist()):
            f = base ** (-2 * n / rot)
            by = min(max((n - first) / (last - first), 0), 1)
            assert math.isclose(got, f * (1 - by) + f / factor * by, rel_tol=1e-12), (rot, n)
        assert math.isclose(m, 0.1 * math.log(factor) + 1)
    # 4096 positions, base 10000: pair 20 turns 36.7 times, pair 21 31.8, so the ramp begins at 20
    fr, _ = dash.rope_freqs(128, scaling="ramp", factor=4.0, device="cpu")
    f, _ = dash.rope_freqs(128, device="cpu")
    assert fr[20] == f[20] and math.isclose(fr[21] / f[21], 1 - 0.75 / 26, rel_tol=1e-12)


def test_ramp_shortened_and_refusals():
    """A factor below one leaves the magnitude at one; the ramp needs a base above one."""
    assert dash.rope_freqs(64, scaling="ramp", factor=0.5, device="cpu")[1] == 1.0
    for base in (1.0, 0.5):
        with pytest.raises(ValueError):
            dash.rope_freqs(64, base=base, scaling="ramp", factor=2.0, device="cpu")
    fr, _ = dash.rope_freqs(64, scaling="ramp", factor=2.0, slow=0.0, device="cpu")
    assert (fr > dash.rope_freqs(64, device="cpu")[0] / 2).all()   # no pair turns less than never
