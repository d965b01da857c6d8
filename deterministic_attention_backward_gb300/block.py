"""A synthetic transformer block, shaped like one decoder layer of an 8B-parameter model
(hidden 4096, 32 query heads, 8 KV heads of 128, SwiGLU MLP of 14336, RMSNorm), timed
forward + backward with this library's attention under each backward schedule.

It gives the end-to-end effect of deterministic attention an in-repo analogue: the DASH
pages report the block-level speedup of their schedules over the deterministic baseline
(technical summary, section 4).  Weights and inputs are random (seeded); there is no
dataset and no optimizer step.  The dense layers use torch matrix products (plumbing around
the measured path); the attention forward and backward run in this library's kernels.

Options put the operators around the attention in their places, forward and backward in this
library's kernels too: rotary positions on the way from the qkv product to the attention, with a norm
of every head of q and k before the turn if asked for, norms fused with the residual joins (with a norm
after each branch as well, if asked for), differential attention with its norm of heads in place of the
attention, the dense products with activation, gate and residual in their epilogues, and after the
backward the clipping of all gradients by their norm.  Without them the block is what it was: no
positions, norms, joins and products in torch operations, gradients as they are.

    python -m deterministic_attention_backward_gb300.block [--seq 8192] [--batch 1]
        [--rotary] [--qk-norm] [--fused-norms] [--post-norms] [--differential] [--fused-dense]
        [--clip]
"""
from __future__ import annotations

import argparse
import json
import statistics


def _attention_function():
    import torch
    import deterministic_attention_backward_gb300 as dash

    class DashAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, causal, schedule):
            o, lse = dash.fwd(q, k, v, causal=causal)
            ctx.save_for_backward(q, k, v, o, lse)
            ctx.causal, ctx.schedule = causal, schedule
            return o

        @staticmethod
        def backward(ctx, do):
            q, k, v, o, lse = ctx.saved_tensors
            dq, dk, dv = dash.bwd(q, k, v, o, do.contiguous(), lse, causal=ctx.causal,
                                  schedule=ctx.schedule)
            return dq, dk, dv, None, None

    return DashAttention


def _operator_functions():
    import torch
    import deterministic_attention_backward_gb300 as dash

    def dense(t):  # a gradient as autograd may hand it in, expanded or transposed
        return None if t is None else t.contiguous()

    class Rotary(torch.autograd.Function):
        """The qkv product's output -> q, k turned and v, each contiguous."""

        @staticmethod
        def forward(ctx, qkv, freqs, q_heads, k_heads, v_heads):
            ctx.save_for_backward(freqs)
            ctx.heads = q_heads, k_heads, v_heads
            return dash.rope_fwd(*Rotary.views(qkv, ctx.heads), inv_freq=freqs)

        @staticmethod
        def backward(ctx, *grads):
            (freqs,) = ctx.saved_tensors
            B, S = grads[0].shape[:2]
            dqkv = grads[0].new_empty(B, S, sum(h * d for h, d in ctx.heads))
            dash.rope_bwd(*map(dense, grads), inv_freq=freqs, out=Rotary.views(dqkv, ctx.heads))
            return dqkv, None, None, None, None

        @staticmethod
        def views(t, heads):
            parts = t.split([h * d for h, d in heads], dim=-1)
            return [p.unflatten(-1, h) for p, h in zip(parts, heads)]

    class NormRotary(torch.autograd.Function):
        """The same with a norm of every head of q and k before the turn."""

        @staticmethod
        def forward(ctx, qkv, wq, wk, freqs, q_heads, k_heads, v_heads):
            ctx.save_for_backward(qkv, wq, wk, freqs)
            ctx.heads = q_heads, k_heads, v_heads
            return dash.rope_norm_fwd(*Rotary.views(qkv, ctx.heads), q_weight=wq, k_weight=wk,
                                      inv_freq=freqs)

        @staticmethod
        def backward(ctx, *grads):
            qkv, wq, wk, freqs = ctx.saved_tensors
            dqkv = torch.empty_like(qkv)
            *_, dwq, dwk = dash.rope_norm_bwd(
                *map(dense, grads), *Rotary.views(qkv, ctx.heads)[:2], q_weight=wq, k_weight=wk,
                inv_freq=freqs, out=Rotary.views(dqkv, ctx.heads))
            return dqkv, dwq, dwk, None, None, None, None

    class Dense(torch.autograd.Function):
        """residual + act(x w), or act(x w) (x w_gate): products with their epilogue."""

        @classmethod
        def call(cls, x, w, w_gate=None, residual=None, act="none"):
            # (in ``forward`` gradients are off whether a backward is to follow or not)
            if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                               for t in (x, w, w_gate, residual)):
                return cls.apply(x, w, w_gate, residual, act)
            return dash.dense_fwd(x, w, act=act, w_gate=w_gate, residual=residual, keep=False)[0]

        @staticmethod
        def forward(ctx, x, w, w_gate, residual, act):
            y, kept = dash.dense_fwd(x, w, act=act, w_gate=w_gate, residual=residual)
            ctx.save_for_backward(x, w, w_gate, kept)
            ctx.act, ctx.joins = act, residual is not None
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, w_gate, kept = ctx.saved_tensors
            dy = dense(dy)
            dx, dw, _, dw_gate, _ = dash.dense_bwd(
                dy, x, w, kept, act=ctx.act, w_gate=w_gate, need_dx=ctx.needs_input_grad[0],
                need_dw=ctx.needs_input_grad[1] or ctx.needs_input_grad[2])
            return dx, dw, dw_gate, dy if ctx.joins else None, None

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            h, rstd = dash.norm_fwd(x, w)
            ctx.save_for_backward(x, rstd, w)
            return h

        @staticmethod
        def backward(ctx, dh):
            return dash.norm_bwd(dense(dh), *ctx.saved_tensors)

    class PreNorm(torch.autograd.Function):
        """x -> x, norm(x): the residual stream's gradient is added inside the norm's."""

        @staticmethod
        def forward(ctx, x, w):
            ctx.set_materialize_grads(False)
            h, rstd = dash.norm_fwd(x, w)
            ctx.save_for_backward(x, rstd, w)
            return x.view_as(x), h

        @staticmethod
        def backward(ctx, dx, dh):
            if dh is None:
                return dx, None
            return dash.norm_bwd(dense(dh), *ctx.saved_tensors, dres=dense(dx))

    class Join(torch.autograd.Function):
        """x, branch -> y = x + norm(branch), and norm(y) where w_next is given."""

        @staticmethod
        def forward(ctx, x, a, w_post, w_next):
            ctx.set_materialize_grads(False)
            y, h, rstd_a, rstd_y = dash.join_fwd(x, a, w_post=w_post, w_next=w_next)
            ctx.save_for_backward(y, a, rstd_a, rstd_y, w_post, w_next)
            return y if w_next is None else (y, h)

        @staticmethod
        def backward(ctx, dy, dh=None):
            y, a, rstd_a, rstd_y, w_post, w_next = ctx.saved_tensors
            if dy is None and dh is None:
                return None, None, None, None
            dx, da, dw_post, _, dw_next = dash.join_bwd(
                dense(dy), dense(dh), y, a, rstd_a, rstd_y, w_post=w_post,
                w_next=None if dh is None else w_next)
            return dx, da, dw_post, dw_next

    class Differential(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, lam, causal):
            rest = q.new_empty(2, *v.shape[:2], q.shape[2] // 2, v.shape[3])
            o, o2, lse = dash.diff_fwd(q, k, v, lam, causal=causal, rest=rest)
            ctx.save_for_backward(q, k, v, o, o2, lse, lam, rest)
            ctx.causal = causal
            return o

        @staticmethod
        def backward(ctx, do):
            q, k, v, o, o2, lse, lam, rest = ctx.saved_tensors
            return *dash.diff_bwd(q, k, v, o, o2, dense(do), lse, lam, causal=ctx.causal,
                                  rest=rest), None

    return Rotary, Norm, PreNorm, Join, Differential, NormRotary, Dense


class Block:
    """Pre-norm decoder block: x + Wo·attn(norm(x)), then + W2·(silu(W1 h) * W3 h).

    ``rotary``: base of rotary positions over the whole of each head of q and k (None: none).
    ``fused_norms``: norms and joins in this library's kernels; ``post_norms``: with them, a norm
    after each branch.  ``differential``: the first map's weight less ``differential`` times the
    second's in every head, the weight learned per head from there on; the projections are the
    same, a head of q or k becomes a pair of half its size, and the heads' outputs are normed
    (the schedule has no meaning then: that backward knows one order only).  ``qk_norm``: with
    rotary, heads of q and k normed before the turn.  ``fused_dense``: products in this library's
    kernels, silu, gate and (without ``fused_norms``, which join by themselves) residual in their
    epilogues."""

    def __init__(self, hidden=4096, heads=32, kv_heads=8, head_dim=128, ffn=14336,
                 device="cuda", seed=0, rotary=None, fused_norms=False, post_norms=False,
                 differential=None, qk_norm=False, fused_dense=False):
        import torch
        if post_norms and not fused_norms:
            raise ValueError("post_norms needs fused_norms")
        if qk_norm and rotary is None:
            raise ValueError("qk_norm needs rotary")
        if differential is not None and head_dim not in (64, 128):
            raise ValueError(f"differential attention needs heads of 64 or 128, got {head_dim}")
        g = torch.Generator(device="cpu").manual_seed(seed)

        def w(n_in, n_out):
            t = torch.randn(n_in, n_out, generator=g, dtype=torch.float32) / n_in ** 0.5
            return t.to(device=device, dtype=torch.bfloat16).requires_grad_()

        self.h, self.hk, self.d = heads, kv_heads, head_dim
        self.wqkv = w(hidden, (heads + 2 * kv_heads) * head_dim)
        self.wo = w(heads * head_dim, hidden)
        self.w1, self.w3, self.w2 = w(hidden, ffn), w(hidden, ffn), w(ffn, hidden)
        self.n1 = torch.ones(hidden, device=device, dtype=torch.bfloat16, requires_grad=True)
        self.n2 = torch.ones(hidden, device=device, dtype=torch.bfloat16, requires_grad=True)
        self.attn = _attention_function()
        (self.Rotary, self.Norm, self.PreNorm, self.Join, self.Differential, self.NormRotary,
         self.Dense) = _operator_functions()
        self.fused_norms, self.fused_dense = fused_norms, fused_dense
        self.p1 = self.p2 = self.lam = self.nh = self.freqs = self.nq = self.nk = None

        def full(n, value, dtype=torch.bfloat16):
            return torch.full((n,), value, device=device, dtype=dtype, requires_grad=True)

        if post_norms:
            self.p1, self.p2 = full(hidden, 1.0), full(hidden, 1.0)
        pair = 1
        if differential is not None:
            pair = 2
            self.lam = full(heads, differential, torch.float32)
            self.nh = full(head_dim, 1.0 - differential)
        # heads of q, k and v as the attention takes them
        self.parts = ((pair * heads, head_dim // pair), (pair * kv_heads, head_dim // pair),
                      (kv_heads, head_dim))
        if rotary is not None:
            from .rope import rope_freqs
            self.freqs, _ = rope_freqs(head_dim // pair, base=rotary, device=device)
        if qk_norm:
            self.nq, self.nk = full(head_dim // pair, 1.0), full(head_dim // pair, 1.0)
        # when a dict: the attention's inputs and output of the last call are kept there, with
        # their gradients retained (q/k/v.grad = dQ/dK/dV, o.grad = the upstream dO)
        self.capture = None

    @staticmethod
    def _rms(x, weight):
        import torch
        xf = x.float()
        return (xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype) * weight

    def __call__(self, x, schedule, causal=True):
        import torch.nn.functional as F
        B, S, _ = x.shape
        if self.fused_norms:
            x, hid = self.PreNorm.apply(x, self.n1)
        else:
            hid = self._rms(x, self.n1)
        fused, joins = self.fused_dense, self.fused_norms
        qkv = self.Dense.call(hid, self.wqkv) if fused else hid @ self.wqkv
        if self.nq is not None:
            q, k, v = self.NormRotary.apply(qkv, self.nq, self.nk, self.freqs, *self.parts)
        elif self.freqs is not None:
            q, k, v = self.Rotary.apply(qkv, self.freqs, *self.parts)
        else:
            q, k, v = (t.reshape(B, S, *heads).contiguous() for t, heads in
                       zip(qkv.split([h * d for h, d in self.parts], dim=-1), self.parts))
        if self.lam is not None:
            o = self.Differential.apply(q, k, v, self.lam, causal)
        else:
            o = self.attn.apply(q, k, v, causal, schedule)
        if self.capture is not None:
            for t in (q, k, v, o):
                t.retain_grad()
            self.capture.update(q=q, k=k, v=v, o=o)
        if self.nh is not None:
            o = self.Norm.apply(o, self.nh)
        o = o.reshape(B, S, self.h * self.d)
        a = self.Dense.call(o, self.wo, residual=None if joins else x) if fused else o @ self.wo
        if joins:
            x, hid = self.Join.apply(x, a, self.p1, self.n2)
        else:
            x = a if fused else x + a
            hid = self._rms(x, self.n2)
        if fused:
            m = self.Dense.call(hid, self.w1, self.w3, act="silu")
            m = self.Dense.call(m, self.w2, residual=None if joins else x)
        else:
            m = (F.silu(hid @ self.w1) * (hid @ self.w3)) @ self.w2
        if joins:
            return self.Join.apply(x, m, self.p2, None)
        return m if fused else x + m

    def parameters(self):
        return [p for p in (self.wqkv, self.wo, self.w1, self.w3, self.w2, self.n1, self.n2,
                            self.p1, self.p2, self.lam, self.nh, self.nq, self.nk)
                if p is not None]

    def clip(self, max_norm):
        """Scale the parameters' gradients in place so that their norm is ``max_norm`` at most: the
        norm they had, an fp32 scalar on the device."""
        import deterministic_attention_backward_gb300 as dash
        return dash.grad_clip([p.grad for p in self.parameters()], max_norm)


def time_block(seq=8192, batch=1, schedules=("atomic", "serial", "shift_fill", "auto"),
               steps=10, warmup=3, causal=True, seed=0, clip=None, **options):
    """Median forward+backward time (ms) of one block per schedule, and each
    deterministic schedule's slowdown against ``atomic``.  ``options`` are those of ``Block``;
    differential attention is timed once, its one order standing for a schedule.  ``clip``: the norm to
    which a step clips its gradients (None: it does not)."""
    import torch
    blk = Block(seed=seed, **options)
    if blk.lam is not None:
        schedules = ("differential",)
    g = torch.Generator(device="cpu").manual_seed(seed + 1)
    x = (torch.randn(batch, seq, 4096, generator=g) * 0.5).to("cuda", torch.bfloat16)
    x.requires_grad_()
    gout = torch.randn(batch, seq, 4096, generator=g).to("cuda", torch.bfloat16)

    def step(sched):
        for p in blk.parameters() + [x]:
            p.grad = None
        out = blk(x, sched, causal)
        out.backward(gout)
        if clip is not None:
            blk.clip(clip)

    res = {}
    for sched in schedules:
        for _ in range(warmup):
            step(sched)
        torch.cuda.synchronize()
        ts = []
        for _ in range(steps):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            step(sched)
            b.record()
            torch.cuda.synchronize()
            ts.append(a.elapsed_time(b))
        res[sched] = statistics.median(ts)
    out = {"block_ms": {k: round(v, 3) for k, v in res.items()}}
    if "atomic" in res:
        out["slowdown_vs_atomic"] = {k: round(v / res["atomic"] - 1, 4)
                                     for k, v in res.items() if k != "atomic"}
    if "serial" in res:
        out["speedup_vs_serial"] = {k: round(res["serial"] / v, 4)
                                    for k, v in res.items() if k not in ("serial", "atomic")}
    out["config"] = {"seq": seq, "batch": batch, "causal": causal, "hidden": 4096,
                     "heads": 32, "kv_heads": 8, "head_dim": 128, "ffn": 14336,
                     "steps": steps, "warmup": warmup, **options}
    if clip is not None:
        out["config"]["clip"] = clip
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--seq", type=int, default=8192)
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--rotary", nargs="?", type=float, const=10000.0, metavar="BASE",
                    help="rotary positions")
    ap.add_argument("--fused-norms", action="store_true",
                    help="norms fused with the residual joins")
    ap.add_argument("--post-norms", action="store_true",
                    help="with --fused-norms, a norm after each branch as well")
    ap.add_argument("--differential", nargs="?", type=float, const=0.8, metavar="WEIGHT",
                    help="differential attention, the second map's weight to begin with")
    ap.add_argument("--qk-norm", action="store_true",
                    help="with --rotary, a norm of every head of q and k before the turn")
    ap.add_argument("--fused-dense", action="store_true",
                    help="products with activation, gate and residual in their epilogue")
    ap.add_argument("--clip", nargs="?", type=float, const=1.0, metavar="NORM",
                    help="clip the gradients to this norm")
    args = ap.parse_args()
    options = {k: v for k, v in (("rotary", args.rotary), ("fused_norms", args.fused_norms),
                                 ("post_norms", args.post_norms),
                                 ("differential", args.differential),
                                 ("qk_norm", args.qk_norm), ("fused_dense", args.fused_dense),
                                 ("clip", args.clip)) if v not in (None, False)}
    if args.post_norms and not args.fused_norms:
        ap.error("--post-norms needs --fused-norms")
    if args.qk_norm and args.rotary is None:
        ap.error("--qk-norm needs --rotary")
    print(json.dumps(time_block(args.seq, args.batch, steps=args.steps, warmup=args.warmup,
                                **options)))


if __name__ == "__main__":
    main()
