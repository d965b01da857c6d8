"""The calls whose kernels are profiled: norms of heads with the turn, products with their epilogue,
clipping."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import deterministic_attention_backward_gb300 as dash  # noqa: E402


def rand(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


inv_freq, _ = dash.rope_freqs(128)
q, k, v = rand(1, 8192, 32, 128), rand(1, 8192, 8, 128), rand(1, 8192, 8, 128)
w = dict(q_weight=rand(128), k_weight=rand(128), inv_freq=inv_freq)
out = dash.rope_norm_fwd(q, k, v, **w)
dash.rope_norm_bwd(*out, q, k, **w)

x, w1, w3, dy = rand(4096, 4096), rand(4096, 7168), rand(4096, 7168), rand(4096, 7168)
y, kept = dash.dense_fwd(x, w1, act="silu", w_gate=w3)
grads = dash.dense_bwd(dy, x, w1, kept, act="silu", w_gate=w3)
dash.dense_fwd(x[:1], w1, act="silu", w_gate=w3, keep=False)

dash.grad_clip([t for t in (*grads, x, dy) if t is not None], 1.0)
torch.cuda.synchronize()
