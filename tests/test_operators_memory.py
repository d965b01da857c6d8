"""Outputs that share memory with what a call reads, or with one another, are refused; views that
lie between one another, and outputs in the place of an input, are not."""
import ctypes
import random

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build
from deterministic_attention_backward_gb300.rope import _PART

BF, F32 = torch.bfloat16, torch.float32
ll = ctypes.c_longlong


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


class Part:
    """A part of a rope call on bf16: tokens [B, S] of `heads` heads of D elements."""

    B, S = 3, 4

    def __init__(self, at, heads, D, strides):
        self.at, self.heads, self.D, self.strides = at, heads, D, strides

    def bytes(self):
        sb, st, sh = self.strides
        return {self.at + 2 * (b * sb + s * st + h * sh + e) for b in range(self.B)
                for s in range(self.S) for h in range(self.heads) for e in range(self.D)}


def rope(L, parts, freq=1 << 40, pos=None, pos_strides=(0, 1)):
    """dash_rope of (in, out) parts that turn nothing, with one more of too many elements: refused
    as unsupported (2) where the others' memory is in order, as invalid (1) where not.  Nothing is
    ever read or written."""
    packed = b"".join(_PART.pack(i.at, o.at, i.heads, i.D, 0, *i.strides, *o.strides)
                      for i, o in parts)
    packed += _PART.pack(1 << 50, 1 << 50, 1, 1 << 28, 0, *[1 << 29] * 6)
    return L.dash_rope(packed, len(parts) + 1, Part.B, Part.S, 2, 0, 0, freq, 1.0, pos, 1,
                       *pos_strides, 0, 0, None)


def test_shared_memory_is_seen(L):
    """Tensors of any strides, near one another: refused exactly where they have an element in
    common."""
    rng, both = random.Random(1), [0, 0]
    base = 1 << 30

    def part(at, heads, D):
        kind = rng.randint(0, 3)
        wide = heads * D + rng.choice([0, 0, rng.randint(0, 40)])
        if kind < 2:    # rows side by side, or at a stride
            strides = (Part.S * wide, wide, D)
        elif kind == 2:  # token slices, heads at a stride
            strides = ((Part.S + rng.randint(0, 2)) * wide * 2, wide * 2, D + rng.randint(0, 5))
        else:
            strides = tuple(rng.randint(0, 60) for _ in range(3))
        return Part(base + 2 * at, heads, D, strides)
    far = 1 << 44
    for _ in range(4000):
        heads, D = rng.randint(1, 3), rng.randint(1, 9)
        a, b = part(rng.randint(0, 200), heads, D), part(rng.randint(0, 200), heads, D)
        want = bool(a.bytes() & b.bytes())
        both[want] += 1
        code = 1 if want else 2
        assert rope(L, [(a, b)]) == (2 if (a.at, a.strides) == (b.at, b.strides) else code)
        one, two = (Part(far + n * far, heads, D, (D * heads * Part.S, D * heads, D))
                    for n in (0, 1))
        assert rope(L, [(one, a), (two, b)]) == code
        assert rope(L, [(one, a), (b, two)]) == code
    assert min(both) > 500


def test_views_of_a_product_lie_apart(L):
    B, S, W = Part.B, Part.S, 6 * 8 + 5
    heads = ((3, 0), (2, 24), (1, 40))

    def views(at):
        return [Part(at + 2 * o, h, 8, (S * W, W, 8)) for h, o in heads[:2]]
    one, two = views(1 << 30), views(1 << 35)
    assert rope(L, list(zip(one, two))) == 2 and rope(L, list(zip(one, one))) == 2
    assert rope(L, [(one[0], one[1]), (two[0], two[1])]) == 2   # between one another
    assert rope(L, [(one[0], two[0]), (one[1], Part(two[0].at + 40, 2, 8, (S * W, W, 8)))]) == 1
    # the frequencies and the positions are read too
    assert rope(L, list(zip(one, two)), freq=two[1].at) == 1
    assert rope(L, list(zip(one, two)), pos=two[0].at + 8 * S, pos_strides=(S, 1)) == 1
    assert rope(L, list(zip(one, two)), pos=two[0].at - 8 * B * S, pos_strides=(S, 1)) == 2


def test_abi_refusals(L):
    M = 1 << 20  # far apart; never dereferenced, as every call is refused
    at = {n: M * (i + 1) for i, n in enumerate(
        ("x", "a", "wp", "g", "wn", "y", "h", "ra", "ry"))}

    def fwd(**moved):
        return L.dash_join_fwd(*{**at, **moved}.values(), 6, 8, 1, (ll * 4)(8, 8, 8, 8), 1.0, 1.0,
                               1e-5, 0, 0, None)
    for out in ("y", "h"):
        for n in ("x", "a"):  # moved on by a row, or back
            assert fwd(**{out: at[n] + 16}) == 1 and fwd(**{out: at[n] - 80}) == 1
        for n, size in (("wp", 16), ("g", 96), ("wn", 16), ("ra", 24), ("ry", 24)):
            assert fwd(**{out: at[n] + size - 2}) == 1 and fwd(**{out: at[n] - 94}) == 1
    assert fwd(y=at["h"] + 94) == 1 and fwd(ra=at["ry"] - 20) == 1 and fwd(ra=at["g"] + 92) == 1
    at = {n: M * (i + 1) for i, n in enumerate(
        ("dy", "dh", "y", "a", "wp", "g", "wn", "ra", "ry", "dx", "da", "dwp", "dg", "dwn"))}

    def bwd(ws=M * 20, **moved):
        return L.dash_join_bwd(*{**at, **moved}.values(), 6, 8, 3, (ll * 6)(*[8] * 6), 1.0, 1.0, 0,
                               0, ws, 1 << 30, None)
    need = L.dash_join_bwd_workspace_bytes(6, 8, 3, 1, 0)
    for out in ("dx", "da"):
        for n in ("dy", "dh", "y", "a"):
            assert bwd(**{out: at[n] + 16}) == 1 and bwd(**{out: at[n] - 80}) == 1
        for n, size in (("wp", 16), ("g", 32), ("wn", 16), ("ra", 24), ("ry", 24), ("dwp", 16),
                        ("dg", 32), ("dwn", 16)):
            assert bwd(**{out: at[n] + size - 2}) == 1 and bwd(**{out: at[n] - 94}) == 1
        assert bwd(ws=at[out] - need // 16 * 16 + 16) == 1
    assert bwd(dwp=at["wp"] + 14) == 1 and bwd(dg=at["dwn"] - 30) == 1 and bwd(ws=at["y"]) == 1

    B, S, H, G, d = 2, 8, 4, 2, 64
    q, kv = B * S * H * 2 * d * 2, B * S * (H // G) * 2 * d * 2

    def diff_fwd(ws=M * 20, **moved):
        p = {**{n: M * (i + 1) for i, n in enumerate(("q", "k", "v", "lam", "o", "o2", "lse"))},
             **moved}
        return L.dash_diff_fwd(*p.values(), B, S, H, G, d, 0.0, 0, 0, 0, ws, 256, None)
    for out in ("o", "o2"):
        for n, size in ((1, q), (2, kv), (3, kv)):
            assert diff_fwd(**{out: M * n + size - 16}) == 1
            assert diff_fwd(**{out: M * n - q + 16}) == 1
        assert diff_fwd(**{out: M * 7 - q + 16}) == 1   # the row sums' memory
    assert diff_fwd(o2=M * 5 + 16) == 1 and diff_fwd(lse=M + q - 4) == 1
    assert diff_fwd(ws=M * 2) == 1 and diff_fwd(ws=M * 6 - 240) == 1

    def diff_bwd(ws=M * 64, **moved):
        p = {**{n: M * (i + 1) for i, n in enumerate(
            ("q", "k", "v", "o", "o2", "do", "lse", "lam", "dq", "dk", "dv", "dlam"))}, **moved}
        return L.dash_diff_bwd(*p.values(), B, S, H, G, d, 0.0, 0, 0, 0, ws, 1 << 30, None)
    for out, mine in (("dq", q), ("dk", kv), ("dv", kv)):
        for n, size in ((1, q), (2, kv), (3, kv), (4, q), (5, q), (6, q), (7, B * 2 * H * S * 4)):
            assert diff_bwd(**{out: M * n + size - 16}) == 1
            assert diff_bwd(**{out: M * n - mine + 16}) == 1
    assert diff_bwd(dk=M * 9 + q - 16) == 1 and diff_bwd(dlam=M * 11 + 2) == 1
    assert diff_bwd(ws=M * 3 + 16) == 1 and diff_bwd(ws=M * 9 + 16) == 1


@pytest.mark.gpu
def test_operators_refuse_shared_memory(L):
    def no(f, *a, **k):
        with pytest.raises((ValueError, dash.DashError)) as err:
            f(*a, **k)
        assert getattr(err.value, "code", 1) == 1
    # norms: rows moved on by one, a weight's memory, two outputs across
    wide, w = torch.ones(9, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    x, up = wide[:8], wide[1:]
    rstd = torch.ones(8, device="cuda")
    no(dash.norm_fwd, x, w, out=up)
    no(dash.join_fwd, x, x.clone(), w_next=w, y=up)
    no(dash.join_fwd, x.clone(), x.clone(), w_next=w, y=x, h=up)
    no(dash.norm_bwd, x, x.clone(), rstd, w, dx=up)
    no(dash.join_bwd, x, x.clone(), x.clone(), x.clone(), None, rstd, w_next=w, da=up)
    no(dash.join_bwd, x, x.clone(), x.clone(), x.clone(), None, rstd, w_next=w, dx=x, da=up)
    no(dash.norm_fwd, x, up.reshape(-1)[32:96], out=up)
    # rope: tokens moved on by one, another part's heads, the positions
    q = torch.ones(1, 9, 4, 64, dtype=F32, device="cuda")
    f, _ = dash.rope_freqs(64)
    no(dash.rope_fwd, q[:, :8], inv_freq=f, out=(q[:, 1:], None, None))
    no(dash.rope_fwd, q[:, :, :2], q[:, :, 2:], inv_freq=f, out=(q[:, :, 1:3], None, None))
    no(dash.rope_fwd, q[:, :, :2], q[:, :, 2:], inv_freq=f, out=(q[:, :, 2:], None, None))
    at = torch.zeros(1 * 9 * 4 * 32, dtype=torch.int64, device="cuda")
    no(dash.rope_fwd, q, inv_freq=f, positions=at[:9], out=(at.view(F32).view(q.shape), None, None))
    # differential attention: a token further, one output across another
    g = torch.zeros(1, 10, 4, 64, dtype=BF, device="cuda")
    q, k, v = g[:, :8], g[:, :8, :2].clone(), torch.zeros(1, 8, 1, 128, dtype=BF, device="cuda")
    lam = torch.zeros(2, device="cuda")
    no(dash.diff_fwd, q, k, v, lam, out=g.view(-1)[256:2304].view(1, 8, 2, 128))
    two = torch.zeros(1, 9, 2, 128, dtype=BF, device="cuda")
    no(dash.diff_fwd, q, k, v, lam, out=two[:, :8], out2=two[:, 1:])
    o, o2, lse = dash.diff_fwd(q, k, v, lam)
    no(dash.diff_bwd, q, k, v, o, o2, two[:, :8], lse, lam, dq=two.view(-1)[8:2056].view(q.shape))


@pytest.mark.gpu
def test_outputs_between_and_in_place(L):
    """Views of one buffer that lie between one another, and in place, are taken, with the bits of
    a call that returns new tensors."""
    g = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.randn(40, 256, generator=g, device="cuda").to(BF)
    x, a, y, h = (buf[:, 64 * i: 64 * i + 64] for i in range(4))
    w = torch.ones(64, dtype=BF, device="cuda")
    want = dash.join_fwd(x, a, w_post=w, w_next=w)
    got = dash.join_fwd(x, a, w_post=w, w_next=w, y=y, h=h)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    y, h, ra, ry = want
    grads = dash.join_bwd(x, a, y, x, ra, ry, w_post=w, w_next=w)
    dx, da = buf[:, 128:192], buf[:, 192:]
    again = dash.join_bwd(x, a, y, x, ra, ry, w_post=w, w_next=w, dx=dx, da=da)
    assert all(p is q or torch.equal(p, q) for p, q in zip(grads, again))
    again = dash.join_bwd(x, a, y, x, ra, ry, w_post=w, w_next=w, dx=a, da=x)
    assert all(p is q or torch.equal(p, q) for p, q in zip(grads, again))
    x, a = (buf[:, 64 * i: 64 * i + 64] for i in (2, 3))
    want = dash.join_fwd(x, a, w_post=w, w_next=w)
    got = dash.join_fwd(x, a, w_post=w, w_next=w, y=a, h=x)  # each in the other's place
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_long_tensors_of_padded_heads(L):
    """Parts of heads of one buffer, whose strides do not flatten: told apart and together over any
    number of tokens."""
    S, W = 200000, 40 * 128 + 24
    strides = (S * W, W, 128)

    def call(at, out):
        parts = [(at, 1 << 50, 0), (out, out, 0)]
        packed = b"".join(_PART.pack(i, o, 3, 64, 0, *strides, *strides) for i, o, _ in parts)
        packed += _PART.pack(1 << 55, 1 << 55, 1, 1 << 28, 0, *[1 << 29] * 6)
        return L.dash_rope(packed, 3, 1, S, 2, 0, 0, 1 << 45, 1.0, None, 1, 0, 1, 0, 0, None)
    base = 1 << 30
    assert call(base, base + 128) == 2              # the other halves of the same heads
    assert call(base, base + 3 * 256) == 2          # the next heads
    assert call(base, base + 126) == 1 and call(base, base + 2 * 256 + 126) == 1
    far = 2 * W * (S - 1)                           # the last token of the one, the first of the other
    assert call(base, base + far + 128) == 2 and call(base, base + far + 256) == 1
    assert call(base + far, base + 128) == 2 and call(base + far, base + 256 - 126) == 1
    import time
    least = 1.0
    for _ in range(50):  # and in a time that does not grow with them (2 us; a walk over tokens 130)
        t = time.perf_counter()
        call(base, base + 128)
        least = min(least, time.perf_counter() - t)
    assert least < 40e-6, least
