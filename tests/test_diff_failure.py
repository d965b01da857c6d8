"""Differential attention's kernels when a block of their input never comes: every bounded wait for
it gives up, the kernels return by themselves, the status word tells, and the next call in the same
workspace is as if nothing had been.  No fault: the loads of a block are left out on purpose."""
import time

import pytest
import torch

import deterministic_attention_backward_gb300 as dash
from deterministic_attention_backward_gb300 import _build

DASH_ERR_TIMEOUT = 4
FWD, DQ, DKV = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return dash.lib()


def test_arguments(L):
    assert L.dash_diff_withhold(-1, 0) == L.dash_diff_withhold(4, 0) == 1
    assert L.dash_diff_withhold(1, -1) == 1 and L.dash_diff_withhold(0, 0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kernel,block", [(FWD, 0), (FWD, 1), (FWD, 7), (DQ, 0), (DQ, 1), (DQ, 4),
                                          (DKV, 0), (DKV, 1), (DKV, 9)])
def test_withheld_block(L, kernel, block, causal, d):
    """At the first block, at one behind it, and behind several tiles or turns of the rings; CTAs
    that need fewer blocks end as always."""
    B, S, H, Hkv = 2, 1000, 24, 12
    g = torch.Generator(device="cuda").manual_seed(block)

    def n(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v, do = n(B, S, 2 * H, d), n(B, S, 2 * Hkv, d), n(B, S, Hkv, 2 * d), n(B, S, H, 2 * d)
    lam = torch.rand(H, generator=g, device="cuda")
    ws = torch.empty(dash.diff_bwd_workspace_bytes(B, S, H, d), dtype=torch.uint8, device="cuda")

    def both():
        o, o2, lse = dash.diff_fwd(q, k, v, lam, causal=causal, workspace=ws, check=kernel != FWD)
        if kernel == FWD and failing:
            return (o, o2, lse)
        return (o, o2, lse, *dash.diff_bwd(q, k, v, o, o2, do, lse, lam, causal=causal,
                                           workspace=ws))
    failing = False
    want = both()
    torch.cuda.synchronize()
    failing = True
    dash.set_wait_limit(0.05)
    assert L.dash_diff_withhold(kernel, block) == 0
    try:
        t0 = time.time()
        both()
        with pytest.raises(dash.DashError) as err:
            dash.status(ws)
        elapsed = time.time() - t0
    finally:
        L.dash_diff_withhold(0, 0)
        dash.set_wait_limit(2.0)
    failing = False
    assert err.value.code == DASH_ERR_TIMEOUT
    # one limit, for all CTAs see the word that the first sets; what is in flight ends within 0.1 s
    assert 0.04 < elapsed < 1.0, elapsed
    again = both()
    dash.status(ws)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
