"""The calls that operators.md profiles: one of each operator, forward and backward, in bf16."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import deterministic_attention_backward_gb300 as dash  # noqa: E402


def rand(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


x, a, dy, dh = (rand(8192, 4096) for _ in range(4))
w = dict(w_post=rand(4096), gate=rand(4096), w_next=rand(4096))
y, h, rstd_a, rstd_y = dash.join_fwd(x, a, **w)
dash.join_bwd(dy, dh, y, a, rstd_a, rstd_y, **w)

inv_freq, _ = dash.rope_freqs(128)
dash.rope_fwd(rand(1, 8192, 32, 128), rand(1, 8192, 8, 128), rand(1, 8192, 8, 128),
              inv_freq=inv_freq)

q, k, v, do = rand(1, 4096, 64, 64), rand(1, 4096, 16, 64), rand(1, 4096, 8, 128), \
    rand(1, 4096, 32, 128)
lam, rest = torch.rand(32, device="cuda"), torch.empty(2, *do.shape, dtype=do.dtype, device="cuda")
o, o2, lse = dash.diff_fwd(q, k, v, lam, rest=rest)
dash.diff_bwd(q, k, v, o, o2, do, lse, lam, rest=rest)
torch.cuda.synchronize()
