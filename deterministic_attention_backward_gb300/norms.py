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
Outputs may be row operands themselves (y and h: x or a; dx and da: dy, dh, y or a), at the same
row stride; beside that no output shares memory with another tensor of the call.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, lib
from ._args import DTYPES, alike, disjoint, run, scratch, tensor

_Strides4, _Strides6 = ctypes.c_longlong * 4, ctypes.c_longlong * 6


def _stride(t, name, like=None):
    """The stride of ``t``'s rows (of ``like``'s type, device and shape); ValueError where the
    dimensions before the last do not flatten to one."""
    if like is not None:
        alike(t, name, like, like.shape)
    C = t.shape[-1]
    if t.is_contiguous():
        return C
    try:
        r = t.view(-1, C)
    except RuntimeError:
        r = None
    if r is None or (C > 1 and r.stride(1) != 1):
        raise ValueError(f"{name} must have contiguous rows at one stride, got strides "
                         f"{tuple(t.stride())}")
    return r.stride(0)


def _out(t, name, like):
    """``_stride`` of a tensor that is written, 0 where there is none."""
    if t is None:
        return 0
    s = _stride(t, name, like)
    if not disjoint(t):
        raise ValueError(f"{name} has elements that share an address")
    return s


def _in_place(outs, ins, weights):
    """Raise ValueError where an output is the memory of another, of an input whose rows lie at
    another stride (both are (tensor, stride of its rows)), or of one of ``weights``, which are
    read after rows have been written."""
    for n, (o, so) in enumerate(outs):
        if o is None or o.numel() == 0:
            continue
        at = o.data_ptr()
        if any(u is not None and u.data_ptr() == at for u, _ in outs[:n]) or \
                any(t is not None and t.data_ptr() == at and st != so for t, st in ins):
            raise ValueError("an output is the memory of another output, or of an input with "
                             "another stride")
        if any(w is not None and w.data_ptr() == at for w in weights):
            raise ValueError("an output is the memory of a weight, a gate or an rstd")


def _weights(x, rows, w_post, gate, w_next):
    """Check the weights against rows of x; returns (their type, rows per gate row)."""
    C, dtype, gate_rows = x.shape[-1], None, rows
    for name, w in (("w_post", w_post), ("gate", gate), ("w_next", w_next)):
        if w is None:
            continue
        if dtype is None:
            dtype = w.dtype if isinstance(w, torch.Tensor) else None
            if dtype != x.dtype and dtype != torch.float32:
                raise ValueError(f"{name} must be {x.dtype} or torch.float32, got {dtype}")
        alike(w, name, x, dtype=dtype)
        if name == "gate" and w.dim() > 1:
            groups = w.numel() // C
            lead = list(w.shape[:-1])
            while lead and lead[-1] == 1:
                lead.pop()
            if w.shape[-1] != C or (rows % groups if groups else rows) or \
                    (x.dim() > 2 and list(x.shape[:len(lead)]) != lead):
                raise ValueError(f"gate {tuple(w.shape)} has no row for each run of consecutive "
                                 f"rows of {tuple(x.shape)}")
            gate_rows = rows // max(groups, 1)
        elif w.dim() != 1 or w.shape[0] != C:
            raise ValueError(f"{name} must have shape {(C,)}, got {tuple(w.shape)}")
        if not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return x.dtype if dtype is None else dtype, gate_rows


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    """A new contiguous tensor of t's shape."""
    return torch.empty_like(t) if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _forward(x, a, w_post, gate, w_next, skip_scale, branch_scale, eps, y, h, stream):
    tensor(x, "x", DTYPES)
    shape = x.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("x needs rows of at least one element")
    C = shape[-1]
    rows = x.numel() // C
    join = a is not None
    xs, as_ = _stride(x, "x"), _stride(a, "branch", x) if join else 0
    wdtype, gate_rows = _weights(x, rows, w_post, gate, w_next)
    if w_next is None:
        h = None
    ys, hs = _out(y, "y", x), _out(h, "h" if join else "out", x)
    if y is not None or h is not None:
        _in_place(((y, ys), (h, hs)), ((x, xs), (a, as_)), (w_post, gate, w_next))

    def launch(handle):
        Y, H, ra, ry = y, h, None, None
        if join and Y is None:
            Y = _like(x)
        if w_next is not None:
            if H is None:
                H = _like(x)
            ry = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        if w_post is not None:
            ra = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        if rows:
            _check(lib().dash_join_fwd(x.data_ptr(), _ptr(a), _ptr(w_post), _ptr(gate),
                                       _ptr(w_next), _ptr(Y) if join else None, _ptr(H), _ptr(ra),
                                       _ptr(ry), rows, C, gate_rows,
                                       _Strides4(xs, as_, ys or C, hs or C), skip_scale,
                                       branch_scale, eps, DTYPES[x.dtype], DTYPES[wdtype],
                                       handle), "dash_join_fwd")
        return Y, H, ra, ry
    return run(x, stream, launch)


def _backward(dy, dh, y, a, rstd_a, rstd_y, w_post, gate, w_next, skip_scale, branch_scale, dx,
              da, workspace, stream):
    join, normed = a is not None, w_next is not None
    base = y if y is not None else a
    tensor(base, "y" if join else "x", DTYPES)
    shape = base.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("y needs rows of at least one element")
    C = shape[-1]
    rows = base.numel() // C
    if normed and (dh is None or y is None or rstd_y is None):
        raise ValueError("the gradient of the norm needs dh, its rows and their rstd")
    if not normed and dy is None:
        raise ValueError("no gradient is given")
    if w_post is not None and rstd_a is None:
        raise ValueError("the gradient of the norm after the branch needs rstd_a")
    ys = 0 if y is None else _stride(y, "y")
    as_ = _stride(a, "branch", base) if join else 0
    dys = 0 if dy is None else _stride(dy, "dy", base)
    dhs = _stride(dh, "dh", base) if normed else 0
    wdtype, gate_rows = _weights(base, rows, w_post, gate, w_next)
    for t, w, n in ((rstd_a, w_post, "rstd_a"), (rstd_y, w_next, "rstd_y")):
        if w is not None:
            alike(t, n, base, shape[:-1], torch.float32)
            if not t.is_contiguous():
                raise ValueError(f"{n} must be contiguous")
    dxs, das = _out(dx, "dx", base), _out(da, "da", base)
    if dx is not None or da is not None:
        _in_place(((dx, dxs), (da, das)), ((dy, dys), (dh, dhs), (y, ys), (a, as_)),
                  (w_post, gate, w_next, rstd_a, rstd_y))

    def launch(handle):
        DX, DA = _like(base) if dx is None else dx, da
        if join and DA is None:
            DA = _like(base)
        dw_post, dgate, dw_next = (None if w is None else torch.empty_like(w)
                                   for w in (w_post, gate, w_next))
        if rows:
            L, dtype = lib(), DTYPES[base.dtype]
            need = L.dash_join_bwd_workspace_bytes(rows, C, gate_rows if gate is not None else 0,
                                                   join, dtype)
            ws = scratch(need or 256, base, workspace)
            _check(L.dash_join_bwd(_ptr(dy), _ptr(dh) if normed else None, _ptr(y), _ptr(a),
                                   _ptr(w_post), _ptr(gate), _ptr(w_next), _ptr(rstd_a),
                                   _ptr(rstd_y), DX.data_ptr(), _ptr(DA), _ptr(dw_post),
                                   _ptr(dgate), _ptr(dw_next), rows, C, gate_rows,
                                   _Strides6(dys, dhs, ys, as_, dxs or C, das or C), skip_scale,
                                   branch_scale, dtype, DTYPES[wdtype], ws.data_ptr(),
                                   ws.numel() * ws.element_size(), handle), "dash_join_bwd")
        else:
            for w in (dw_post, dgate, dw_next):
                if w is not None:
                    w.zero_()
        return DX, DA if join else None, dw_post, dgate, dw_next
    return run(base, stream, launch)


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
    it serving the same number of consecutive rows of x ([B, C] or [B, 1, C] for x [B, S, C])."""
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
