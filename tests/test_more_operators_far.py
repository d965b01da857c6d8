"""The block's further operators on tensors of more than 2^31 elements: offsets pass 32 bits."""
import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    yield
    torch.cuda.empty_cache()


def filled(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(n, dtype=BF, device="cuda")
    for at in range(0, n, 1 << 28):
        part = t[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return t


def test_heads():
    """The last tokens of a long batch give the bits that they give alone."""
    B, S, H, D = 1, 4300, 4096, 128  # 2.25e9 elements
    x = filled(B * S * H * D, 0).view(B, S, H, D)
    w = torch.linspace(0.5, 1.5, D, device="cuda").to(BF)
    f, _ = dash.rope_freqs(D)
    y = dash.rope_norm_fwd(x, q_weight=w, inv_freq=f)[0]
    last = dash.rope_norm_fwd(x[:, -7:], q_weight=w, inv_freq=f, start=S - 7)[0]
    assert torch.equal(y[:, -7:], last)
    dx, _, _, dw, _ = dash.rope_norm_bwd(y, None, None, x, q_weight=w, inv_freq=f, out=(y, None, None))
    # y is the gradient of |y|^2 / 2, which of a head does not depend on its length: dx is small
    # against y rstd; and w dw sums |y|^2 over all heads: D each for w = 1
    part = dash.rope_norm_bwd(last, None, None, x[:, -7:].contiguous(), q_weight=w, inv_freq=f,
                              start=S - 7)
    assert torch.equal(dx[:, -7:], part[0])
    # E[x^2] = 1 up to 2^-10 over 1.7e7 heads, dw = sum of w x^2: rounding to bf16 on top
    assert ((dw.double() / (w.double() * S * H) - 1).abs() <= 2.0 ** -9 + 2.0 ** -8).all()


def test_dense():
    """Rows and outputs beyond 2^31 elements: the last rows against the same rows alone."""
    M, K, N = 140000, 136, 16384  # 2.29e9 outputs
    x, w = filled(M * K, 1).view(M, K), filled(K * N, 2).view(K, N)
    y, kept = dash.dense_fwd(x, w, act="silu", check=True)
    few, kept_few = dash.dense_fwd(x[-300:], w, act="silu")
    assert torch.equal(y[-300:], few)
    dx, dw, *_ = dash.dense_bwd(y, x, w, kept, act="silu", check=True)
    part = dash.dense_bwd(few, x[-300:], w, kept_few, act="silu")
    # the same products, perhaps split otherwise: fp32 sums in another order
    err = (dx[-300:].double() - part[0].double()).norm() / part[0].double().norm()
    assert err <= 2.0 ** -8
    del y, kept
    head = slice(0, 64)  # dw's first columns from 64 bits, by rows of x
    ref = torch.zeros(K, 64, dtype=torch.float64, device="cuda")
    for at in range(0, M, 20000):
        X = x[at:at + 20000].double()
        z = X @ w[:, head].double()
        s = torch.sigmoid(z)
        dy = (z * s).to(BF).double()
        ref += X.t() @ (dy * (s + z * s * (1 - s)))
    err = (dw[:, head].double() - ref).norm() / ref.norm()
    # dy, dz and dw are rounded: 2^-8 / sqrt 3 each
    assert err <= 3 * 2.0 ** -8 / 3 ** 0.5


def test_grads():
    n = (1 << 31) + 12345
    g = filled(n, 3)
    norm = dash.grad_norm([g])
    ref = sum(float(g[at:at + (1 << 27)].double().square().sum()) for at in range(0, n, 1 << 27)) ** 0.5
    assert abs(float(norm) - ref) <= 2.0 ** -17 * ref
    tail = g[-5000:].clone()
    dash.grad_clip([g], 0.5 * ref)
    assert ((g[-5000:].double() - 0.5 * tail.double()).abs() <=
            (2.0 ** -9 + 2.0 ** -16) * 0.5 * tail.double().abs()).all()


def test_sizes_that_do_not_fit():
    """Sizes behind 2^31 come from views of one element; what would wrap is refused, nothing is formed."""
    one = torch.ones(1, 1, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="2\\^30"):
        dash.dense_fwd(one.expand(4, 1), one.expand(1, 2 ** 32 + 5))
    with pytest.raises(ValueError, match="2\\^30"):
        dash.dense_fwd(one.expand(2 ** 32 + 5, 1), one)
    f, _ = dash.rope_freqs(2)
    far = torch.ones(1, 1, 2, dtype=BF, device="cuda").expand(2 ** 32 + 5, 1, 2)
    for call in (dash.rope_norm_fwd, dash.rope_fwd):
        with pytest.raises(ValueError, match="2\\^31"):
            call(far, inv_freq=f)
        with pytest.raises(ValueError, match="2\\^31"):
            call(far[:1], None, far[:1, :, :1].expand(1, 2 ** 32 + 5, 1), inv_freq=f)
