"""Differential attention: the difference of two softmax maps with a learned weight, forward and
deterministic backward.

    o, o2, lse = diff_fwd(q, k, v, lam, causal=True)
    dq, dk, dv, dlam = diff_bwd(q, k, v, o, o2, do, lse, lam, causal=True)

    O = softmax(scale Q1 K1^T) V - lam softmax(scale Q2 K2^T) V

q [B,S,2H,d], k [B,S,2Hkv,d], v [B,S,Hkv,2d] bf16 with d = 32 or 64: head pair h reads the query
maps 2h and 2h+1 and shares the keys and values of pair h // (H / Hkv).  These are the projections
of attention with H heads of 2d, viewed with heads of d for q and k.  lam [H] or [B,S,H], bf16
or fp32.  o2 (the second map's output) and lse [B,2H,S] are what the backward needs besides o.

A training step should keep what o and o2 lose by their rounding too, two bf16 tensors more:

    rest = torch.empty(2, *o_shape, dtype=torch.bfloat16, device=q.device)
    o, o2, lse = diff_fwd(q, k, v, lam, causal=True, rest=rest)
    dq, dk, dv, dlam = diff_bwd(q, k, v, o, o2, do, lse, lam, causal=True, rest=rest)

for the row terms D = dO . Om of dQ: off by 2.4e-3 to 3.3e-3 of its norm with rest, without it by
2.5e-3 for flat maps and up to 8e-3 where a few keys dominate them.
"""
from __future__ import annotations

import torch

from . import _check, lib, status
from ._args import alike, apart, contiguous, run, scratch, tensor

_BF16 = (torch.bfloat16,)


def _dims(q, k, v, lam):
    tensor(q, "q", _BF16)
    if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q and v must be [B, S, heads, d]")
    B, S, H2, d = q.shape
    Hkv = v.shape[2]
    if H2 % 2 or Hkv == 0 or (H2 // 2) % Hkv:
        raise ValueError(f"q {tuple(q.shape)} has no whole group of head pairs for each head of "
                         f"v {tuple(v.shape)}")
    alike(k, "k", q, (B, S, 2 * Hkv, d))
    alike(v, "v", q, (B, S, Hkv, 2 * d))
    H = H2 // 2
    tensor(lam, "lam", (torch.bfloat16, torch.float32))
    if lam.device != q.device:
        raise ValueError(f"lam is on {lam.device}, expected {q.device}")
    if lam.shape != (H,) and lam.shape != (B, S, H):
        raise ValueError(f"lam must be {(H,)} or {(B, S, H)}, got {tuple(lam.shape)}")
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (lam, "lam")):
        contiguous(t, n)
    return B, S, H, Hkv, d


def _given(t, name, like, shape, dtype=None):
    """An output or a saved tensor that the caller hands in."""
    alike(t, name, like, shape, dtype)
    contiguous(t, name)


def diff_fwd_workspace_bytes(B: int, S: int, H: int, d: int) -> int:
    """Workspace bytes of ``diff_fwd`` for H head pairs of maps of d elements (0: unsupported)."""
    return int(lib().dash_diff_fwd_workspace_bytes(B, S, H, d))


def diff_bwd_workspace_bytes(B: int, S: int, H: int, d: int) -> int:
    """Workspace bytes of ``diff_bwd`` for H head pairs of maps of d elements (0: unsupported)."""
    return int(lib().dash_diff_bwd_workspace_bytes(B, S, H, d))


def diff_fwd(q, k, v, lam, causal: bool = False, scale: float | None = None, out=None, out2=None,
             lse=None, workspace=None, stream=None, check: bool = False, rest=None):
    """Forward: returns (O [B,S,H,2d], O2 = softmax(Q2 K2^T) V of the same shape, LSE [B,2H,S]).
    ``rest`` ([2,B,S,H,2d] bf16) receives what O and O2 lose by their rounding, for ``diff_bwd``.
    A ``workspace`` serves one call at a time."""
    B, S, H, Hkv, d = _dims(q, k, v, lam)
    shape = (B, S, H, 2 * d)
    if out is not None:
        _given(out, "out", q, shape)
    if out2 is not None:
        _given(out2, "out2", q, shape)
    if lse is not None:
        _given(lse, "lse", q, (B, 2 * H, S), torch.float32)
    if rest is not None:
        _given(rest, "rest", q, (2, *shape))
    if out is not None or out2 is not None or lse is not None or rest is not None:
        apart((out, out2, lse, rest), (q, k, v, lam))

    def launch(handle):
        o = torch.empty(shape, dtype=q.dtype, device=q.device) if out is None else out
        o2 = torch.empty_like(o) if out2 is None else out2
        l = lse if lse is not None else torch.empty((B, 2 * H, S), dtype=torch.float32,
                                                    device=q.device)
        if B and S:
            L = lib()
            ws = scratch(L.dash_diff_fwd_workspace_bytes(B, S, H, d) or 256, q, workspace)
            _check(L.dash_diff_fwd_rest(q.data_ptr(), k.data_ptr(), v.data_ptr(), lam.data_ptr(),
                                        o.data_ptr(), o2.data_ptr(),
                                        None if rest is None else rest.data_ptr(), l.data_ptr(),
                                        B, S, H, H // Hkv, d, scale or 0.0, bool(causal),
                                        2 * (lam.dtype == torch.float32), lam.dim() == 3,
                                        ws.data_ptr(), ws.numel() * ws.element_size(), handle),
                   "dash_diff_fwd")
            if check:
                status(ws, torch.cuda.current_stream())
        return o, o2, l
    return run(q, stream, launch)


def diff_bwd(q, k, v, o, o2, do, lse, lam, causal: bool = False, scale: float | None = None,
             dq=None, dk=None, dv=None, dlam=None, workspace=None, stream=None,
             check: bool = False, rest=None):
    """Backward: returns (dQ, dK, dV, dlam), bit-identical on every run.  ``rest``: what the
    forward wrote there."""
    B, S, H, Hkv, d = _dims(q, k, v, lam)
    shape = (B, S, H, 2 * d)
    _given(o, "o", q, shape)
    _given(o2, "o2", q, shape)
    _given(do, "do", q, shape)
    _given(lse, "lse", q, (B, 2 * H, S), torch.float32)
    if rest is not None:
        _given(rest, "rest", q, (2, *shape))
    for t, n, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v), (dlam, "dlam", lam)):
        if t is not None:
            _given(t, n, q, like.shape, like.dtype)
    if dq is not None or dk is not None or dv is not None or dlam is not None:
        apart((dq, dk, dv, dlam), (q, k, v, o, o2, do, lse, lam, rest))

    def launch(handle):
        gq, gk, gv, gl = (torch.empty_like(like) if t is None else t
                          for t, like in ((dq, q), (dk, k), (dv, v), (dlam, lam)))
        if not (B and S):
            gl.zero_()
            return gq, gk, gv, gl
        L = lib()
        ws = scratch(L.dash_diff_bwd_workspace_bytes(B, S, H, d) or 256, q, workspace)
        _check(L.dash_diff_bwd_rest(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                    o2.data_ptr(), None if rest is None else rest.data_ptr(),
                                    do.data_ptr(), lse.data_ptr(), lam.data_ptr(), gq.data_ptr(),
                                    gk.data_ptr(), gv.data_ptr(), gl.data_ptr(), B, S, H,
                                    H // Hkv, d, scale or 0.0, bool(causal),
                                    2 * (lam.dtype == torch.float32), lam.dim() == 3,
                                    ws.data_ptr(), ws.numel() * ws.element_size(), handle),
               "dash_diff_bwd")
        if check:
            status(ws, torch.cuda.current_stream())
        return gq, gk, gv, gl
    return run(q, stream, launch)
