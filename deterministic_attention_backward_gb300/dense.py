"""Matrix products with bias, activation, gate and residual in their epilogue, forward and backward.

    y, kept = dense_fwd(x, w, bias, act="gelu", residual=r)                  # y = r + gelu(x w + bias)
    y, kept = dense_fwd(x, w, act="silu", w_gate=u)                          # y = silu(x w) (x u)
    dx, dw, dbias, dw_gate, dbias_gate = dense_bwd(dy, x, w, kept, act="silu", w_gate=u)

x [..., K] are rows of one stride, bf16 or fp16; w [K, N] (and w_gate) has either dimension contiguous
(the transpose of a weight stored [N, K] too).  Sums are fp32, in an order that the sizes fix: the same
bits on every run.  Sizes and addresses may be any; what does not lie on 16 bytes is copied into the
workspace first.
"""
from __future__ import annotations

import struct

import torch

from . import _check, lib, status
from ._args import DTYPES, alike, contiguous, run, scratch, tensor
from .norms import _out, _ptr, _stride

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_TYPES = (torch.bfloat16, torch.float16)
_KN, _NK = 0, 1

# dash_dense_fwd_t: x, w, w_gate, bias, bias_gate, residual, y, z, gate; their strides; M, K, N,
# order, act, dtype
_FWD = struct.Struct("@9P5q6i")
# dash_dense_bwd_t: dy, x, w, w_gate, z, gate, dx, dw, dw_gate, dbias, dbias_gate; their strides; ...
_BWD = struct.Struct("@11P7q6i")


def _order(w, name, order=None):
    """(order, row stride) of a weight [K, N]: rows of N elements, or of K."""
    K, N = w.shape
    sk, sn = w.stride()
    if order is None:
        order = _NK if (sk == 1 or K == 1) and (sn != 1 or N == 1) and not (K == 1 and sn == 1) \
            else _KN
    if order == _KN and (sn == 1 or N == 1):
        return order, sk if K > 1 else N
    if order == _NK and (sk == 1 or K == 1):
        return order, sn if N > 1 else K
    raise ValueError(f"{name} must have one dimension contiguous (the same as w's), got strides "
                     f"{tuple(w.stride())}")


def _weights(x, w, w_gate, act):
    """Check x and the weights; returns (rows, K, N, order, stride, the gate's stride)."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    if x.dim() < 1 or not isinstance(w, torch.Tensor) or w.dim() != 2 or \
            w.shape[0] != x.shape[-1] or not w.numel():
        raise ValueError(f"w must be [K, N] for rows x of K elements, got "
                         f"{tuple(getattr(w, 'shape', ()))} for {tuple(x.shape)}")
    alike(w, "w", x)
    K, N = w.shape
    order, ws = _order(w, "w")
    gs = 0
    if w_gate is not None:
        alike(w_gate, "w_gate", x, w.shape)
        _, gs = _order(w_gate, "w_gate", order)
    rows = x.numel() // K
    if max(rows, K, N) > 1 << 30:
        raise ValueError(f"products of {rows} x {K} x {N} are not taken, 2^30 at most")
    return rows, K, N, order, ws, gs


def _kept_bytes(rows, N):
    return 3 * rows * ((N + 15) // 16 * 16)


def _biases(x, N, w_gate, bias, bias_gate):
    for b, n in ((bias, "bias"), (bias_gate, "bias_gate")):
        if b is not None:
            alike(b, n, x, (N,))
            contiguous(b, n)
    if bias_gate is not None and w_gate is None:
        raise ValueError("bias_gate needs w_gate")


def _fwd_args(x, w, bias, act, w_gate, bias_gate, residual, out, keep):
    """Check the forward's arguments; returns what fills its arguments."""
    tensor(x, "x", _TYPES)
    rows, K, N, order, ws, gs = _weights(x, w, w_gate, act)
    xs = _stride(x, "x")
    _biases(x, N, w_gate, bias, bias_gate)
    shape = (*x.shape[:-1], N)
    rs = ys = 0
    if residual is not None:
        alike(residual, "residual", x, shape)
        rs = _stride(residual, "residual")
    if out is not None:
        alike(out, "out", x, shape)
        ys = _out(out, "out", out)
    return rows, K, N, order, shape, (xs, ws, gs, rs, ys or N)


def dense_fwd_workspace_bytes(x, w, *, w_gate=None, residual=None, out=None) -> int:
    """Workspace bytes of ``dense_fwd`` for these tensors (as they lie in memory)."""
    rows, K, N, order, shape, strides = _fwd_args(x, w, None, "none", w_gate, None, residual, out, False)
    if rows == 0:
        return 0
    y = 1 << 20 if out is None else out.data_ptr()  # (a new one lies on 16 bytes)
    a = _FWD.pack(x.data_ptr(), w.data_ptr(), _ptr(w_gate) or 0, 0, 0, _ptr(residual) or 0, y, 0, 0,
                  *strides, rows, K, N, order, 0, DTYPES[x.dtype])
    return int(lib().dash_dense_fwd_workspace_bytes(a))


def dense_fwd(x, w, bias=None, *, act: str = "none", w_gate=None, bias_gate=None, residual=None,
              keep: bool = True, out=None, workspace=None, stream=None, check: bool = False):
    """y = residual + act(x w + bias), or residual + act(x w + bias) (x w_gate + bias_gate): returns
    (y [..., N], kept).  ``kept`` is what ``dense_bwd`` needs besides, x w + bias and, where there is a
    gate, x w_gate + bias_gate: each value rounded to 24 bits in a uint8 tensor of the library's layout; None
    for ``act`` "none" without a gate, or ``keep=False``.  ``out`` may be the residual itself (at its strides).  A
    ``workspace`` serves one call at a time."""
    rows, K, N, order, shape, strides = _fwd_args(x, w, bias, act, w_gate, bias_gate, residual, out,
                                                  keep)

    def launch(handle):
        y = torch.empty(shape, dtype=x.dtype, device=x.device) if out is None else out
        kept = None
        if keep and (act != "none" or w_gate is not None):
            kept = torch.empty((1 if w_gate is None else 2, _kept_bytes(rows, N)),
                               dtype=torch.uint8, device=x.device)
        if rows == 0:
            return y, kept
        z = _ptr(kept) or 0
        g = z + kept.shape[1] if z and w_gate is not None else 0
        L = lib()
        a = _FWD.pack(x.data_ptr(), w.data_ptr(), _ptr(w_gate) or 0, _ptr(bias) or 0,
                      _ptr(bias_gate) or 0, _ptr(residual) or 0, y.data_ptr(), z, g, *strides,
                      rows, K, N, order, ACTIVATIONS[act], DTYPES[x.dtype])
        ws = scratch(L.dash_dense_fwd_workspace_bytes(a) or 256, x, workspace)
        _check(L.dash_dense_fwd(a, ws.data_ptr(), ws.numel() * ws.element_size(), handle),
               "dash_dense_fwd")
        if check:
            status(ws, torch.cuda.current_stream())
        return y, kept
    return run(x, stream, launch)


def _bwd_args(dy, x, w, kept, act, w_gate, bias, bias_gate, dx, dw, dw_gate):
    tensor(x, "x", _TYPES)
    rows, K, N, order, ws, gs = _weights(x, w, w_gate, act)
    shape = (*x.shape[:-1], N)
    alike(dy, "dy", x, shape)
    xs, dys = _stride(x, "x"), _stride(dy, "dy")
    _biases(x, N, w_gate, bias, bias_gate)
    gated = w_gate is not None
    if act != "none" or gated:
        if kept is None:
            raise ValueError("the gradient needs what the forward kept")
        alike(kept, "kept", x, (1 + gated, _kept_bytes(rows, N)), torch.uint8)
        contiguous(kept, "kept")
    dxs = 0 if dx is None else _out(dx, "dx", x)
    dws = dgs = 0
    for t, n in ((dw, "dw"), (dw_gate, "dw_gate")):
        if t is not None:
            if n == "dw_gate" and not gated:
                raise ValueError("dw_gate needs w_gate")
            alike(t, n, x, w.shape)
            _, s = _order(t, n, order)
            if s < (N if order == _KN else K):
                raise ValueError(f"{n} has elements that share an address")
            dws, dgs = (s, dgs) if n == "dw" else (dws, s)
    line = N if order == _KN else K
    return rows, K, N, order, (dys, xs, ws, gs, dxs or K, dws or line, dgs or line)


def _terms(terms, rows):
    if terms not in (None, 1, 2):
        raise ValueError(f"terms must be 1, 2 or None, got {terms}")
    if terms == 2 and rows > 1 << 29:
        raise ValueError(f"two terms of {rows} rows are not taken, 2^29 at most")
    return terms or 0


def _bwd_pack(dy, x, w, kept, act, w_gate, dx, dw, dw_gate, db, dbg, rows, K, N, order, strides):
    gated = w_gate is not None
    z = g = 0
    if act != "none" or gated:
        z = kept.data_ptr()
        g = z + kept.shape[1] if gated else 0
    return _BWD.pack(dy.data_ptr(), x.data_ptr(), w.data_ptr(), _ptr(w_gate) or 0, z, g, dx, dw,
                     dw_gate, db, dbg, *strides, rows, K, N, order, ACTIVATIONS[act],
                     DTYPES[x.dtype])


def dense_bwd_workspace_bytes(dy, x, w, kept=None, *, act: str = "none", w_gate=None, bias=None,
                              bias_gate=None, dx=None, dw=None, dw_gate=None, terms=None) -> int:
    """Workspace bytes of ``dense_bwd`` for these tensors (as they lie in memory), all gradients
    asked for."""
    args = _bwd_args(dy, x, w, kept, act, w_gate, bias, bias_gate, dx, dw, dw_gate)
    terms = _terms(terms, args[0])
    if args[0] == 0:
        return 256

    def at(t, wanted=True):  # (a new one lies on 16 bytes)
        return t.data_ptr() if t is not None else 1 << 20 if wanted else 0
    a = _bwd_pack(dy, x, w, kept, act, w_gate, at(dx), at(dw), at(dw_gate, w_gate is not None),
                  0 if bias is None else at(None), 0 if bias_gate is None else at(None), *args)
    return int(lib().dash_dense_bwd_terms_workspace_bytes(a, terms))


def dense_bwd(dy, x, w, kept=None, *, act: str = "none", w_gate=None, bias=None, bias_gate=None,
              need_dx: bool = True, need_dw: bool = True, dx=None, dw=None, dw_gate=None, terms=None,
              workspace=None, stream=None, check: bool = False):
    """Gradient of ``dense_fwd``: returns (dx, dw, dbias, dw_gate, dbias_gate), None for what is not
    there (``need_dx``, ``need_dw``: not asked for; of the biases only their presence matters).  dw and
    dw_gate have their weight's layout in memory.  The residual's gradient is dy itself.

    The products take dz = dy act'(z) (and the gate's) rounded to x's type, which is off by as much as
    the results' own rounding; ``terms=2`` multiplies what that loses too, which doubles the products.
    Left to itself the call takes two terms of up to 2^16 elements of dz, so ``terms=1`` or ``2`` is
    for programs whose results must not depend on that.  Infinities and NaN come out as of one term."""
    args = _bwd_args(dy, x, w, kept, act, w_gate, bias, bias_gate, dx, dw, dw_gate)
    rows, K, N, order, strides = args
    terms = _terms(terms, rows)
    gated = w_gate is not None

    def launch(handle):
        def weight(given):
            if given is not None:
                return given
            if order == _KN:
                return torch.empty((K, N), dtype=x.dtype, device=x.device)
            return torch.empty((N, K), dtype=x.dtype, device=x.device).t()
        DX = DW = DG = None
        if need_dx:
            DX = torch.empty(x.shape, dtype=x.dtype, device=x.device) if dx is None else dx
        if need_dw:
            DW = weight(dw)
            DG = weight(dw_gate) if gated else None
        db, dbg = (None if b is None else torch.empty(N, dtype=x.dtype, device=x.device)
                   for b in (bias, bias_gate))
        if rows == 0:
            for t in (DW, db, DG, dbg):
                if t is not None:
                    t.zero_()
            return DX, DW, db, DG, dbg
        L = lib()
        a = _bwd_pack(dy, x, w, kept, act, w_gate, *(_ptr(t) or 0 for t in (DX, DW, DG, db, dbg)),
                      *args)
        ws = scratch(L.dash_dense_bwd_terms_workspace_bytes(a, terms) or 256, x, workspace)
        _check(L.dash_dense_bwd_terms(a, terms, ws.data_ptr(), ws.numel() * ws.element_size(), handle),
               "dash_dense_bwd_terms")
        if check:
            status(ws, torch.cuda.current_stream())
        return DX, DW, db, DG, dbg
    return run(x, stream, launch)
