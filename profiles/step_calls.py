"""The calls whose kernels are profiled, one by its name: norms of heads with the turn, products with their
epilogue, clipping."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import deterministic_attention_backward_gb300 as dash  # noqa: E402


def rand(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


def heads(back):
    inv_freq, _ = dash.rope_freqs(128)
    q, k, v = rand(1, 8192, 32, 128), rand(1, 8192, 8, 128), rand(1, 8192, 8, 128)
    w = dict(q_weight=rand(128), k_weight=rand(128), inv_freq=inv_freq)
    if back:
        dash.rope_norm_bwd(q, k, v, *map(torch.clone, (q, k)), **w)
    else:
        dash.rope_norm_fwd(q, k, v, **w)


def dense(M, K, N, back, **wanted):
    x, w1, w3, dy = rand(M, K), rand(K, N), rand(K, N), rand(M, N)
    y, kept = dash.dense_fwd(x, w1, act="silu", w_gate=w3, keep=back or M > 1)
    if back:
        dash.dense_bwd(dy, x, w1, kept, act="silu", w_gate=w3, **wanted)


def clip():
    grads = [rand(4096, 4096), rand(4096, 7168), rand(4096, 7168), rand(4096, 7168), rand(4096, 4096)]
    dash.grad_clip(grads, 1.0)


CALLS = {
    "heads_fwd": lambda: heads(False),
    "heads_bwd": lambda: heads(True),
    "dense_fwd": lambda: dense(4096, 4096, 7168, False),
    "dense_dx": lambda: dense(4096, 4096, 7168, True, need_dw=False),
    "dense_dw": lambda: dense(4096, 4096, 7168, True, need_dx=False),
    "dense_row": lambda: dense(1, 4096, 7168, False),
    "dense_row_dx": lambda: dense(1, 4096, 7168, True, need_dw=False),
    "clip": clip,
}

if __name__ == "__main__":
    CALLS[sys.argv[1]]()
    torch.cuda.synchronize()
