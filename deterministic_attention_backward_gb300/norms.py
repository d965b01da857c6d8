"""Root-mean-square norm of rows, and the join of a residual stream with a branch between two
norms, forward and backward.

    h, rstd = norm_fwd(x, w)
    dx, dw = norm_bwd(dh, x, rstd, w, dres=dx_of_the_residual_stream)

    y, h, rstd_a, rstd_y = join_fwd(x, a, w_post=w1, gate=g, w_next=w2, branch_scale=0.5)
    dx, da, dw1, dg, dw2 = join_bwd(dy, dh, y, a, rstd_a, rstd_y, w_post=w1, gate=g, w_next=w2,
                                    branch_scale=0.5)

    y = skip_scale x + branch_scale gate (a rstd(a) w_post),    h = y rstd(y) w_next

Rows are the last dimension of tensors of any shape (the rest must flatten to one row stride),
bf16, fp16 or fp32; weights of the rows' type or fp32.  The weight gradients are deterministic.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _workspace, lib
from ._args import DTYPES, disjoint, placed, shaped, tensor


def _rows(t, name, like=None):
    """``t`` as [rows, C] without a copy; ValueError where it has no such form."""
    if like is None:
        tensor(t, name, dtypes=DTYPES)
        if t.dim() < 1 or t.shape[-1] == 0:
            raise ValueError(f"{name} needs rows of at least one element")
    else:
        tensor(t, name, like=like)
        shaped(t, name, like.shape)
    try:
        r = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(-1, t.shape[-1])
    except RuntimeError:
        r = None
    if r is None or (r.shape[-1] > 1 and r.stride(-1) != 1):
        raise ValueError(f"{name} must have contiguous rows at one stride, got strides "
                         f"{tuple(t.stride())}")
    return r


def _written(t, name, like):
    r = _rows(t, name, like)
    if not disjoint(r):
        raise ValueError(f"{name} has elements that share an address")
    return r


def _weights(x, rows, **weights):
    """Check the weights against rows of x; returns (their type, rows per gate row)."""
    C, dtype, gate_rows = x.shape[-1], None, rows
    for name, w in weights.items():
        if w is None:
            continue
        tensor(w, name, dtypes=(x.dtype, torch.float32))
        if w.device != x.device:
            raise ValueError(f"{name} is on {w.device}, expected {x.device}")
        if dtype is not None and w.dtype != dtype:
            raise ValueError(f"{name} is {w.dtype}, the other weights {dtype}")
        dtype = w.dtype
        if name == "gate" and w.dim() > 1:
            groups = w.numel() // C if C else 0
            if w.shape[-1] != C or groups == 0 or rows % groups:
                raise ValueError(f"gate {tuple(w.shape)} does not divide {rows} rows of {C}")
            gate_rows = rows // groups
        else:
            shaped(w, name, (C,))
        if not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return x.dtype if dtype is None else dtype, gate_rows


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stride(r):
    return 0 if r is None else r.stride(0)


def _forward(x, a, w_post, gate, w_next, skip_scale, branch_scale, eps, y, h, stream):
    xr = _rows(x, "x")
    ar = None if a is None else _rows(a, "branch", x)
    rows, C = xr.shape
    wdtype, gate_rows = _weights(x, rows, w_post=w_post, gate=gate, w_next=w_next)
    for t, n in ((y, "y"), (h, "h" if a is not None else "out")):
        if t is not None:
            _written(t, n, x)
    with placed(x, stream):
        new = dict(dtype=x.dtype, device=x.device)
        if a is not None and y is None:
            y = torch.empty(x.shape, **new)
        if w_next is not None and h is None:
            h = torch.empty(x.shape, **new)
        rstd = dict(dtype=torch.float32, device=x.device)
        rstd_a = torch.empty(x.shape[:-1], **rstd) if w_post is not None else None
        rstd_y = torch.empty(x.shape[:-1], **rstd) if w_next is not None else None
        if w_next is None:
            h = None
        if rows:
            yr = None if a is None else _rows(y, "y", x)
            hr = None if h is None else _rows(h, "h", x)
            strides = (ctypes.c_longlong * 4)(_stride(xr), _stride(ar), _stride(yr), _stride(hr))
            code = lib().dash_join_fwd(x.data_ptr(), _ptr(a), _ptr(w_post), _ptr(gate),
                                       _ptr(w_next), _ptr(yr), _ptr(hr), _ptr(rstd_a),
                                       _ptr(rstd_y), rows, C, gate_rows, strides,
                                       float(skip_scale), float(branch_scale), float(eps),
                                       DTYPES[x.dtype], DTYPES[wdtype],
                                       torch.cuda.current_stream().cuda_stream)
            _check(code, "dash_join_fwd")
    return y, h, rstd_a, rstd_y


def _backward(dy, dh, y, a, rstd_a, rstd_y, w_post, gate, w_next, skip_scale, branch_scale, dx,
              da, workspace, stream):
    base = y if y is not None else a
    yr = None if y is None else _rows(y, "y" if a is not None else "x")
    ar = None if a is None else _rows(a, "branch", base)
    rows, C = (yr if yr is not None else ar).shape
    wdtype, gate_rows = _weights(base, rows, w_post=w_post, gate=gate, w_next=w_next)
    dyr = None if dy is None else _rows(dy, "dy", base)
    if w_next is not None and (dh is None or y is None or rstd_y is None):
        raise ValueError("the gradient of the norm needs dh, its rows and their rstd")
    dhr = None if w_next is None else _rows(dh, "dh", base)
    if w_next is None and dy is None:
        raise ValueError("no gradient is given")
    if w_post is not None and rstd_a is None:
        raise ValueError("the gradient of the norm after the branch needs rstd_a")
    for t, w, n in ((rstd_a, w_post, "rstd_a"), (rstd_y, w_next, "rstd_y")):
        if w is not None:
            tensor(t, n, like=base, dtypes=(torch.float32,))
            shaped(t, n, base.shape[:-1])
            if not t.is_contiguous():
                raise ValueError(f"{n} must be contiguous")
    for t, n in ((dx, "dx"), (da, "da")):
        if t is not None:
            _written(t, n, base)
    with placed(base, stream):
        dx = torch.empty(base.shape, dtype=base.dtype, device=base.device) if dx is None else dx
        if a is not None and da is None:
            da = torch.empty(base.shape, dtype=base.dtype, device=base.device)
        dw_post, dgate, dw_next = (None if w is None else torch.empty_like(w)
                                   for w in (w_post, gate, w_next))
        if rows == 0:
            for w in (dw_post, dgate, dw_next):
                if w is not None:
                    w.zero_()
            return dx, da, dw_post, dgate, dw_next
        dxr = _rows(dx, "dx", base)
        dar = None if a is None else _rows(da, "da", base)
        need = lib().dash_join_bwd_workspace_bytes(rows, C, gate_rows if gate is not None else 0,
                                                   int(a is not None), DTYPES[base.dtype])
        ws = _workspace(int(need) or 256, base.device, workspace)
        strides = (ctypes.c_longlong * 6)(*(_stride(r) for r in (dyr, dhr, yr, ar, dxr, dar)))
        code = lib().dash_join_bwd(_ptr(dy), _ptr(dh) if w_next is not None else None, _ptr(y),
                                   _ptr(a), _ptr(w_post), _ptr(gate), _ptr(w_next), _ptr(rstd_a),
                                   _ptr(rstd_y), dx.data_ptr(), _ptr(da), _ptr(dw_post),
                                   _ptr(dgate), _ptr(dw_next), rows, C, gate_rows, strides,
                                   float(skip_scale), float(branch_scale), DTYPES[base.dtype],
                                   DTYPES[wdtype], ws.data_ptr(), ws.numel() * ws.element_size(),
                                   torch.cuda.current_stream().cuda_stream)
        _check(code, "dash_join_bwd")
    return dx, da, dw_post, dgate, dw_next


def norm_bwd_workspace_bytes(rows: int, C: int, dtype) -> int:
    """Workspace bytes of ``norm_bwd`` for ``rows`` rows of ``C`` elements."""
    return int(lib().dash_join_bwd_workspace_bytes(rows, C, 0, 0, DTYPES[dtype]))


def join_bwd_workspace_bytes(rows: int, C: int, dtype, gate_rows: int = 0) -> int:
    """Workspace bytes of ``join_bwd``; ``gate_rows``: consecutive rows that share a row of the
    gate (0 without a gate)."""
    return int(lib().dash_join_bwd_workspace_bytes(rows, C, gate_rows, 1, DTYPES[dtype]))


def norm_fwd(x, w, *, eps: float = 1e-5, out=None, stream=None):
    """h = x rstd(x) w over the last dimension: returns (h, rstd), rstd fp32 for ``norm_bwd``."""
    if w is None:
        raise ValueError("norm_fwd needs a weight")
    _, h, _, rstd = _forward(x, None, None, None, w, 1.0, 1.0, eps, None, out, stream)
    return h, rstd


def norm_bwd(dh, x, rstd, w, *, dres=None, dx=None, workspace=None, stream=None):
    """Gradient of ``norm_fwd``: returns (dx, dw).  ``dres``, a gradient that reaches x beside
    the norm (the residual stream's), is added to dx."""
    if w is None:
        raise ValueError("norm_bwd needs a weight")
    dx, _, _, _, dw = _backward(dres, dh, x, None, None, rstd, None, None, w, 1.0, 1.0, dx, None,
                                workspace, stream)
    return dx, dw


def join_fwd(x, a, *, w_post=None, gate=None, w_next=None, skip_scale: float = 1.0,
             branch_scale: float = 1.0, eps: float = 1e-5, y=None, h=None, stream=None):
    """y = skip_scale x + branch_scale gate (a rstd(a) w_post), h = y rstd(y) w_next: returns
    (y, h, rstd_a, rstd_y).  Without ``w_post`` the branch is not normed, without ``gate`` it is
    not gated, without ``w_next`` there is no h.  ``gate`` is [C], or [..., C] with every row of
    it serving the same number of consecutive rows of x ([B, C] for x [B, S, C])."""
    if a is None:
        raise ValueError("join_fwd needs a branch")
    return _forward(x, a, w_post, gate, w_next, skip_scale, branch_scale, eps, y, h, stream)


def join_bwd(dy, dh, y, a, rstd_a=None, rstd_y=None, *, w_post=None, gate=None, w_next=None,
             skip_scale: float = 1.0, branch_scale: float = 1.0, dx=None, da=None, workspace=None,
             stream=None):
    """Gradient of ``join_fwd`` from those of its outputs y (None where nothing else uses it)
    and h: returns (dx, da, dw_post, dgate, dw_next), None for a weight that is not there."""
    if a is None:
        raise ValueError("join_bwd needs the branch")
    return _backward(dy, dh, y, a, rstd_a, rstd_y, w_post, gate, w_next, skip_scale, branch_scale,
                     dx, da, workspace, stream)
