"""The norm over many gradients and clipping by it, against 64 bits.

Tolerances.  A thread adds the squares of at most 512 elements of a chunk in fp32, by four partial sums:
the sum is off by at most 140 2^-24 of itself, the norm by half that, and by its rounding to fp32.  The
factor takes that and three roundings of 2^-24, a scaled gradient one more and its rounding, eps / 2."""
import math

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build
from deterministic_attention_backward_gb300.grads import _GRAD

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
gpu = pytest.mark.gpu
NORM = 72 * 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def make(shape, dtype, seed, by=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)


def norm_of(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def check(got, grads, max_norm, norm, eps=1e-6):
    by = min(1.0, max_norm / (norm + eps))
    for g, t in zip(got, grads):
        fi = torch.finfo(t.dtype)
        ref = t.double() * by
        tol = (NORM + 5 * 2.0 ** -24 + fi.eps / 2) * ref.abs() + fi.smallest_normal * fi.eps
        assert ((g.double() - ref).abs() <= tol).all()


def test_abi_refusals(L):
    at = 1 << 20  # never dereferenced: every call below is refused first

    def pack(*rows):
        return b"".join(_GRAD.pack(*r, 0) for r in rows)
    one = pack((at, at, 16, 0))
    ok = dict(g=one, n=1, max_norm=1.0, eps=0.0, given=0, norm=8 * at, ws=16 * at, bytes=1 << 20)

    def clip(**k):
        k = {**ok, **k}
        return L.dash_grad_clip(k["g"], k["n"], k["max_norm"], k["eps"], k["given"] or None,
                                k["norm"] or None, k["ws"] or None, k["bytes"], None)
    for bad in (dict(n=-1), dict(g=None), dict(g=pack((0, at, 16, 0))), dict(g=pack((at, 0, 16, 0))),
                dict(g=pack((at, at, -1, 0))), dict(g=pack((at, at, 1, 3))),
                dict(g=pack((at + 1, at + 1, 1, 0))), dict(g=pack((at + 2, at + 2, 1, 2))),
                dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=-1.0), dict(eps=math.nan),
                dict(norm=0), dict(norm=8 * at + 2), dict(given=2), dict(norm=at), dict(ws=at),
                dict(norm=16 * at), dict(g=one * 2, n=2),
                dict(g=pack((at, 2 * at, 16, 0), (2 * at + 30, 3 * at, 16, 0)), n=2),
                dict(g=pack((at, at + 2, 16, 0)))):
        assert clip(**bad) == 1, bad
    assert clip(g=pack((at, at, 1 << 46, 0))) == 2
    assert clip(ws=0) == 5 and clip(bytes=100) == 5 and clip(ws=16 * at + 8) == 5
    assert L.dash_grad_norm(one, 1, None, 16 * at, 1 << 20, None) == 1
    assert L.dash_grad_norm(one, 1, at + 4, 16 * at, 1 << 20, None) == 1
    assert L.dash_grad_norm(one, 1, 8 * at, at, 1 << 20, None) == 1
    assert L.dash_grad_norm(one, 1, 8 * at, None, 0, None) == 5
    assert L.dash_grad_norm_workspace_bytes(-1) == 0


SETS = {
    "one": [((1,), F32)],
    "few": [((5,), BF), ((3, 7), F32), ((0,), BF), ((64, 65), HF), ((1 << 14,), BF)],
    "layer": [((512, 1536), BF), ((512, 512), BF), ((512, 777), BF), ((777, 512), BF), ((512,), F32)],
    "large": [((4096, 4099), BF), ((3 << 20,), F32), ((8191,), HF), ((8193,), F32)],
    "many": [((1 + 37 * i % 900,), (BF, HF, F32)[i % 3]) for i in range(1300)],
}


@gpu
@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(L, name):
    grads = [make(s, t, i, 0.1 + i % 3) for i, (s, t) in enumerate(SETS[name])]
    ref = norm_of(grads)
    norm = dash.grad_norm(grads)
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - ref) <= (NORM + 2.0 ** -24) * ref
    assert torch.equal(norm, dash.grad_norm(grads))
    mine = [t.clone() for t in grads]
    # within the limit: untouched
    assert torch.equal(dash.grad_clip(mine, 2 * ref), norm)
    assert all(torch.equal(a, b) for a, b in zip(mine, grads))
    for limit in (0.37 * ref, 0.0):
        out = [torch.full_like(t, 7.0) for t in grads]
        got = dash.grad_clip(grads, limit, out=out)
        assert torch.equal(got, norm)
        check(out, grads, limit, ref)
        mine = [t.clone() for t in grads]
        dash.grad_clip(mine, limit)
        assert all(torch.equal(a, b) for a, b in zip(mine, out))
    out = [torch.full_like(t, 7.0) for t in grads]
    dash.grad_clip(grads, math.inf, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, grads))
    # a norm over more than these
    more = torch.tensor(3 * ref, device="cuda")
    out = [torch.empty_like(t) for t in grads]
    assert dash.grad_clip(grads, ref, norm=more, out=out) is more
    check(out, grads, ref, float(more))


@gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 5), (0, 1), (7, 0)])
def test_offsets(L, dtype, a, b):
    """Gradients in a flat buffer, off 16 bytes, to others; nothing beside them is written."""
    for n in (1, 5, 63, 20000):
        flat = make((n + 16,), dtype, n)
        to = torch.full((n + 16,), 7.0, dtype=dtype, device="cuda")
        g, o = flat[a:a + n], to[b:b + n]
        ref = norm_of([g])
        norm = dash.grad_clip([g], ref / 3, out=[o])
        assert abs(float(norm) - ref) <= (NORM + 2.0 ** -24) * ref
        check([o], [g], ref / 3, ref)
        assert (to[:b] == 7).all() and (to[b + n:] == 7).all()
        keep = flat.clone()
        dash.grad_clip(g, ref / 3)
        assert torch.equal(g, o)
        assert torch.equal(flat[:a], keep[:a]) and torch.equal(flat[a + n:], keep[a + n:])


@gpu
def test_transposed_and_absent(L):
    w = make((100, 40), F32, 0)
    t = w.t()
    ref = norm_of([w])
    assert abs(float(dash.grad_norm([None, t])) - ref) <= (NORM + 2.0 ** -24) * ref
    p = make((4, 6, 8), BF, 1).permute(2, 0, 1)
    mine = [t.clone(memory_format=torch.preserve_format), None, p.clone(memory_format=torch.preserve_format)]
    ref = norm_of([t, p])
    dash.grad_clip(mine, 0.5 * ref)
    check([mine[0], mine[2]], [t, p], 0.5 * ref, ref)
    for bad in (w[:, :39], w[::2], w[:1].expand(5, 40)):
        with pytest.raises(ValueError):
            dash.grad_norm([bad])


@gpu
@pytest.mark.parametrize("by", [2.0 ** 100, 2.0 ** 70, 2.0 ** -70, 2.0 ** -120])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_magnitudes_whose_squares_fp32_does_not_hold(L, dtype, by):
    g = (make((70001,), F32, 3) * by).to(dtype)
    small = make((70001,), dtype, 4)
    for grads in ([g], [g, small], [g, torch.zeros_like(g)]):
        ref = norm_of(grads)
        assert abs(float(dash.grad_norm(grads)) - ref) <= (NORM + 2.0 ** -24) * ref
    assert float(dash.grad_norm([torch.zeros_like(g)])) == 0.0
    out = [torch.empty_like(g)]
    dash.grad_clip([g], 1.0, out=out)
    # the norm is finite, the factor may be as small as 2^-110 and is held with its full precision
    check(out, [g], 1.0, norm_of([g]))


@gpu
def test_special_values(L):
    g, h = make((1000,), BF, 0), make((3000,), F32, 1)
    g[77] = math.inf
    assert float(dash.grad_norm([g, h])) == math.inf
    out = [torch.empty_like(g), torch.empty_like(h)]
    assert float(dash.grad_clip([g, h], 1.0, out=out)) == math.inf
    assert (out[1] == 0).all() and out[0].isnan().sum() == 1 and (out[0] == 0).sum() == 999
    g[78] = math.nan
    assert math.isnan(float(dash.grad_clip([g, h], 1.0)))
    assert g.isnan().all() and h.isnan().all()
    z = torch.zeros(10, device="cuda")
    assert float(dash.grad_clip([z, torch.empty(0, device="cuda")], 1.0)) == 0 and (z == 0).all()
    assert float(dash.grad_clip([z], 0.0, eps=0.0)) == 0 and (z == 0).all()
    e = torch.empty(0, device="cuda")
    assert float(dash.grad_norm([e])) == 0 and float(dash.grad_clip([e], 1.0)) == 0


@gpu
def test_streams_graphs_and_refusals(L):
    grads = [make((300, 200), BF, 0), make((5000,), F32, 1)]
    ref = dash.grad_norm(grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in grads]
    norm = dash.grad_clip(grads, 1.0, out=out, stream=s)
    s.synchronize()
    assert torch.equal(norm, ref)
    ws = torch.empty(dash.grad_norm_workspace_bytes(2), dtype=torch.uint8, device="cuda").fill_(255)
    mine = [t.clone() for t in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = dash.grad_clip(mine, 1.0, workspace=ws)
    for by in (1.0, 3.0):
        for m, t in zip(mine, grads):
            m.copy_(t * by)
        want = [torch.empty_like(t) for t in grads]
        n = dash.grad_clip([m.clone() for m in mine], 1.0, out=want)
        graph.replay()
        assert torch.equal(norm, n) and all(torch.equal(a, b) for a, b in zip(mine, want))
    g = grads[0]
    for bad in (lambda: dash.grad_norm([]), lambda: dash.grad_norm([None]),
                lambda: dash.grad_norm([g.cpu()]), lambda: dash.grad_norm([g, g.cpu()]),
                lambda: dash.grad_norm([g.long()]), lambda: dash.grad_norm([g, "x"]),
                lambda: dash.grad_clip([g], -1.0), lambda: dash.grad_clip([g], math.nan),
                lambda: dash.grad_clip([g], 1.0, eps=-1.0), lambda: dash.grad_clip([g], 1.0, out=[]),
                lambda: dash.grad_clip([g], 1.0, out=[g.float()]),
                lambda: dash.grad_clip([g], 1.0, out=[torch.empty(200, 300, dtype=BF, device="cuda").t()]),
                lambda: dash.grad_clip([g], 1.0, norm=torch.ones(2, device="cuda")),
                lambda: dash.grad_norm([g], out=torch.empty((), dtype=BF, device="cuda")),
                lambda: dash.grad_norm([g], workspace=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dash.DashError):
        dash.grad_clip([g, g], 1.0)
    with pytest.raises(dash.DashError):
        dash.grad_clip([g, g[:10]], 1.0, out=[torch.empty_like(g), g[10:20]])


@gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_bits_do_not_depend_on_the_place_in_memory(L, dtype):
    """A gradient in a flat buffer gives the same norm wherever it begins: its elements are added in the
    order of their numbers.  One element so large that what is added to it by itself is lost, the others so
    that it matters which of them are."""
    bits = {BF: 8, HF: 11, F32: 24}[dtype]
    for n in (1, 7, 8, 9, 100, 2047, 2048, 2049, 8192, 20001, 300000):
        for at in {0, 1, n // 2, n - 1}:
            # squares of 2^-25 and less beside 1: every one is lost alone
            src = make((n,), F32, n).abs().clamp(0.25, 1) * 2.0 ** -12.5
            src[min(at, n - 1)] = 1.0 + 2.0 ** (1 - bits)
            src = src.to(dtype)
            got = set()
            for offset in range(9):
                flat = torch.full((n + 16,), 7.0, dtype=dtype, device="cuda")
                flat[offset:offset + n] = src
                norm = dash.grad_norm([flat[offset:offset + n]])
                got.add(float(norm))
                out = torch.empty_like(flat)[offset:offset + n]
                again = dash.grad_clip([flat[offset:offset + n]], 0.5, out=[out])
                assert torch.equal(again, norm)
            assert len(got) == 1, (n, at, got)
            ref = norm_of([src])
            assert abs(got.pop() - ref) <= (NORM + 2.0 ** -24) * ref


@gpu
def test_zeros_are_read_once(L):
    """The norm of zeros (as gradients of a table's rows are that a step has not met) takes no longer than
    that of other values; the tensor is larger than L2."""
    z = torch.zeros(1 << 28, device="cuda")
    r = make((1 << 28,), F32, 0)
    time = {}
    for name, g in (("zeros", [z]), ("values", [r])):
        out, ws = torch.empty((), device="cuda"), torch.empty(
            dash.grad_norm_workspace_bytes(1), dtype=torch.uint8, device="cuda")
        runs = []
        for _ in range(12):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(4):
                dash.grad_norm(g, out=out, workspace=ws)
            end.record()
            end.synchronize()
            runs.append(start.elapsed_time(end))
        time[name] = sorted(runs)[len(runs) // 2]
    assert time["zeros"] < 1.3 * time["values"], time
    assert float(dash.grad_norm([z])) == 0.0
    # signed zeros, and a single value of the smallest among them
    z.neg_()
    assert float(dash.grad_norm([z])) == 0.0
    for at in (0, 12345678, z.numel() - 1):
        z[at] = 2.0 ** -149
        assert float(dash.grad_norm([z])) == 2.0 ** -149
        z[at] = 0.0


def test_workspace_of_the_largest_counts(L):
    for n in (0, 1, 512, 513, (1 << 31) - 512, (1 << 31) - 511, (1 << 31) - 1):
        assert L.dash_grad_norm_workspace_bytes(n) == ((n + 511) // 512 + 1) * 608 * 8, n


@gpu
def test_an_infinite_limit_clips_nothing(L):
    g, h = make((1000,), BF, 0), make((3000,), F32, 1)
    g[77], h[5] = math.inf, -math.inf
    mine, out = [g.clone(), h.clone()], [torch.empty_like(g), torch.empty_like(h)]
    assert float(dash.grad_clip(mine, math.inf)) == math.inf
    dash.grad_clip([g, h], math.inf, out=out)
    dash.grad_clip(mine, math.inf, norm=torch.tensor(math.inf, device="cuda"))
    for a, b, ref in zip(mine, out, (g, h)):
        assert torch.equal(a, ref) and torch.equal(b, ref)
    g[78] = math.nan
    assert math.isnan(float(dash.grad_clip([g, h], math.inf)))
    assert g.isnan().all() and h.isnan().all()
