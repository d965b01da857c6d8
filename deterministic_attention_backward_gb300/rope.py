"""Rotary positions for the heads of a qkv product, forward and backward.

    inv_freq, magnitude = rope_freqs(128, base=10000.0)
    q, k, v = rope_fwd(q, k, v, inv_freq=inv_freq)          # turned, contiguous; v copied
    rope_bwd(dq, dk, dv, inv_freq=inv_freq, out=views_of_dqkv)

    q, k, v = rope_norm_fwd(q, k, v, q_weight=wq, k_weight=wk, inv_freq=inv_freq)
    dq, dk, dv, dwq, dwk = rope_norm_bwd(dq, dk, dv, q, k, q_weight=wq, k_weight=wk, inv_freq=inv_freq)

Heads are [B, S, H, D] (or packed [T, H, D]); any strides with contiguous heads, bf16, fp16 or
fp32.  One kernel launch turns q and k and copies v; ``rope_norm_fwd`` norms every head of q and k
(root mean square over the head, times a weight) in the same launch before it turns them.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _check, lib
from ._args import DTYPES, alike, contiguous, disjoint, run, scratch, tensor

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = ("none", "linear", "base", "ramp")

# dash_rope_part_t: in, out, heads, D, turn, in_stride[3], out_stride[3]
_PART = struct.Struct("@PPiii4x6q")


def rope_freqs(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_len: int = 4096, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Frequencies (radians per position, float64 [rot/2] on ``device``) and magnitude of the
    rotary turn of the first ``rot`` elements of a head: pair p turns by base^(-2p/rot) per
    position, scaled for contexts ``factor`` times the trained one:

    - ``"linear"``: every frequency divided by ``factor``
    - ``"base"``: the base raised by factor^(rot/(rot-2)), so that the slowest pair is divided
      by ``factor`` and the fastest kept
    - ``"ramp"``: pairs that turn more than ``fast`` times over ``original_len`` positions kept,
      pairs that turn less than ``slow`` times divided by ``factor``, a linear ramp over the pair
      index between, from the floor of the index at ``fast`` turns to the ceiling of that at
      ``slow`` (YaRN, arXiv 2309.00071); magnitude 0.1 ln(factor) + 1, 1 for factors below one
    """
    if rot <= 0 or rot % 2:
        raise ValueError(f"rot must be positive and even, got {rot}")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor([base ** (-2.0 * p / rot) for p in range(rot // 2)], dtype=torch.float64)
    magnitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if original_len <= 0 or not fast > slow or not base > 1:
            raise ValueError("ramp wants original_len > 0, fast > slow and base > 1")

        def index(turns):  # of the pair that turns so often over original_len positions
            if turns <= 0:
                return rot - 1
            return rot * math.log(original_len / (2.0 * math.pi * turns)) / (2.0 * math.log(base))
        first = max(math.floor(index(fast)), 0)
        last = min(math.ceil(index(slow)), rot - 1)
        p = torch.arange(rot // 2, dtype=torch.float64)
        by = ((p - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
        f = f * (1.0 - by) + f / factor * by
        magnitude = 0.1 * math.log(max(factor, 1.0)) + 1.0
    return f.to(device), magnitude


def _frequencies(q, inv_freq, layout):
    """Check q, the layout and the frequencies; returns (tokens, B, S, the elements that turn)."""
    tensor(q, "q", DTYPES)
    dims = q.dim()
    if dims != 4 and dims != 3:
        raise ValueError(f"heads are [B, S, H, D] or [T, H, D], got {tuple(q.shape)}")
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    alike(inv_freq, "inv_freq", q, dtype=torch.float64)
    rot = 2 * inv_freq.numel()
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or not 0 < rot <= 1024:
        raise ValueError("inv_freq must be contiguous float64 [rot/2], rot <= 1024")
    tokens = q.shape[:-2]
    B, S = tokens if dims == 4 else (1, tokens[0])
    if B * S >= 1 << 31:  # (C integers wrap)
        raise ValueError(f"q {tuple(q.shape)} has 2^31 tokens or more")
    return tokens, B, S, rot


def _heads(t, name, q, i, tokens, rot):
    """Check heads that go with q (part i of q, k, v)."""
    shape = t.shape
    if i:
        alike(t, name, q)
        if shape[:-2] != tokens or t.dim() != q.dim():
            raise ValueError(f"{name} {tuple(shape)} does not go with q {tuple(q.shape)}")
    D = shape[-1]
    if D * shape[-2] >= 1 << 31:
        raise ValueError(f"{name} {tuple(shape)} has 2^31 elements a token or more")
    if i < 2 and D < rot:
        raise ValueError(f"{name} has heads of {D}, fewer than the {rot} that turn")
    if D > 1 and t.stride(-1) != 1:
        raise ValueError(f"the elements of a head of {name} must be contiguous")


def _parts(parts, out, q, tokens, rot):
    """Check the tensors that are read and those that are given to be written; returns the latter."""
    given = out is not None
    out = tuple(out) if given else (None, None, None)
    if len(out) != len(parts):
        raise ValueError(f"out must hold {len(parts)} tensors")
    for i, t in enumerate(parts):
        if t is None:
            continue
        name, shape = "qkv"[i], t.shape
        _heads(t, name, q, i, tokens, rot)
        o = out[i]
        if o is not None:
            name = f"out[{i}]"
            alike(o, name, q, shape)
            if shape[-1] > 1 and o.stride(-1) != 1:
                raise ValueError(f"the elements of a head of {name} must be contiguous")
            if not disjoint(o):
                raise ValueError(f"{name} has elements that share an address")
    if given:  # in place: its own input, as it lies
        at = [t.data_ptr() if t is not None and t.numel() else None for t in parts + out]
        for i, o in enumerate(out, len(parts)):
            if at[i] is not None and at[i] in at[:i] + at[i + 1:] and (
                    at.count(at[i]) > 2 or at[i - len(parts)] != at[i] or
                    o.stride() != parts[i - len(parts)].stride()):
                raise ValueError(f"out[{i - len(parts)}] is the memory of another tensor")
    return out


def _positions(positions, start, q, tokens, S):
    """(pointer, 64 bits, stride of a batch, stride of a token)"""
    if positions is None:
        if not -2 ** 63 <= start <= 2 ** 63 - S:
            raise ValueError(f"positions from {start} on do not fit 64 bits")
        return None, 0, 0, 0
    tensor(positions, "positions", (torch.int32, torch.int64))
    if positions.device != q.device:
        raise ValueError(f"positions are on {positions.device}, the heads on {q.device}")
    if positions.shape != tokens and positions.shape != tokens[-1:]:
        raise ValueError(f"positions must be {tuple(tokens)} or {tuple(tokens[-1:])}, got "
                         f"{tuple(positions.shape)}")
    return (positions.data_ptr(), int(positions.dtype == torch.int64),
            positions.stride(0) if positions.dim() == 2 else 0, positions.stride(-1))


def _new(t):
    return torch.empty_like(t) if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _pack(t, o, turn):
    ti, to = t.stride(), o.stride()
    if t.dim() == 3:
        ti, to = (0, *ti), (0, *to)
    return _PART.pack(t.data_ptr(), o.data_ptr(), t.shape[-2], t.shape[-1], int(turn), ti[0],
                      ti[1], ti[2], to[0], to[1], to[2])


def _rope(parts, inv_freq, magnitude, positions, start, layout, out, stream, back):
    q = parts[0]
    tokens, B, S, rot = _frequencies(q, inv_freq, layout)
    out = _parts(parts, out, q, tokens, rot)
    where, pos64, pb, pt = _positions(positions, start, q, tokens, S)

    def launch(handle):
        res, packed = [], []
        for t, o in zip(parts, out):
            if t is None:
                res.append(None)
                continue
            if o is None:
                o = _new(t)
            res.append(o)
            if t.numel():
                packed.append(_pack(t, o, len(res) < 3))
        if packed:
            _check(lib().dash_rope(b"".join(packed), len(packed), B, S, rot, LAYOUTS[layout],
                                   DTYPES[q.dtype], inv_freq.data_ptr(), magnitude, where, pos64,
                                   pb, pt, start, back, handle), "dash_rope")
        return tuple(res)
    return run(q, stream, launch)


def rope_fwd(q, k=None, v=None, *, inv_freq, magnitude: float = 1.0, positions=None,
             start: int = 0, layout: str = "half", out=None, stream=None):
    """Turn the heads of q (and k) with their tokens' positions and copy v: returns (q, k, v),
    contiguous unless ``out`` gives the tensors to write (strided ones too; an input itself is
    turned in place; beside that they share no memory with a tensor of the call).  Position of
    token s: ``positions`` (int32 or int64, [B, S] or [S]; [T] for packed heads), or
    ``start`` + s."""
    return _rope((q, k, v), inv_freq, magnitude, positions, start, layout, out, stream, False)


def rope_bwd(dq, dk=None, dv=None, *, inv_freq, magnitude: float = 1.0, positions=None,
             start: int = 0, layout: str = "half", out=None, stream=None):
    """Gradient of ``rope_fwd``: from the gradients of its outputs those of its inputs
    (``out``: for example views of the qkv product's gradient)."""
    return _rope((dq, dk, dv), inv_freq, magnitude, positions, start, layout, out, stream, True)


def _head_weights(q, k, v, q_weight, k_weight):
    """Check the norms' weights and the heads' size; returns the weights' type."""
    dtype = None
    for name, w, t in (("q_weight", q_weight, q), ("k_weight", k_weight, k)):
        if w is None:
            continue
        if t is None:
            raise ValueError(f"{name} without {name[0]}")
        if dtype is None:
            dtype = w.dtype if isinstance(w, torch.Tensor) else None
            if dtype != q.dtype and dtype != torch.float32:
                raise ValueError(f"{name} must be {q.dtype} or torch.float32, got {dtype}")
        alike(w, name, q, t.shape[-1:], dtype)
        contiguous(w, name)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is not None and t.shape[-1] > 512:
            raise ValueError(f"{name} has heads of {t.shape[-1]}, 512 at most are taken")
    return q.dtype if dtype is None else dtype


def _two(a, b):
    return (ctypes.c_void_p * 2)(None if a is None else a.data_ptr(),
                                 None if b is None else b.data_ptr())


def rope_norm_fwd(q, k=None, v=None, *, q_weight=None, k_weight=None, inv_freq, eps: float = 1e-5,
                  magnitude: float = 1.0, positions=None, start: int = 0, layout: str = "half",
                  out=None, stream=None):
    """Norm every head of q (and k) over its elements, x rstd(x) weight (weights [D] of the heads'
    type or fp32; None: ones), turn it with its token's position, copy v: returns (q, k, v).  The
    other arguments as in ``rope_fwd``; heads of 512 elements at most."""
    parts = (q, k, v)
    tokens, B, S, rot = _frequencies(q, inv_freq, layout)
    out = _parts(parts, out, q, tokens, rot)
    wtype = _head_weights(q, k, v, q_weight, k_weight)
    where, pos64, pb, pt = _positions(positions, start, q, tokens, S)

    def launch(handle):
        res, packed, weights = [], [], []
        for i, (t, o) in enumerate(zip(parts, out)):
            if t is None:
                res.append(None)
                continue
            res.append(_new(t) if o is None else o)
            if t.numel():
                packed.append(_pack(t, res[-1], i < 2))
                if i < 2:
                    weights.append((q_weight, k_weight)[i])
        if weights:
            _check(lib().dash_rope_norm_fwd(b"".join(packed), len(packed),
                                            _two(*weights, *[None] * (2 - len(weights))), B, S, rot,
                                            LAYOUTS[layout], DTYPES[q.dtype], DTYPES[wtype],
                                            inv_freq.data_ptr(), magnitude, eps, where, pos64, pb, pt,
                                            start, handle), "dash_rope_norm_fwd")
        elif packed:  # heads of v alone
            res[2].copy_(v)
        return tuple(res)
    return run(q, stream, launch)


def rope_norm_bwd_workspace_bytes(D: int) -> int:
    """Workspace bytes of ``rope_norm_bwd`` for heads of D elements (of q or k, whichever has a
    weight; none is needed where neither has)."""
    return int(lib().dash_rope_norm_bwd_workspace_bytes(D))


def rope_norm_bwd(dq, dk, dv, q, k=None, *, q_weight=None, k_weight=None, inv_freq,
                  eps: float = 1e-5, magnitude: float = 1.0, positions=None, start: int = 0,
                  layout: str = "half", out=None, workspace=None, stream=None):
    """Gradient of ``rope_norm_fwd`` from the gradients of its outputs and its inputs q and k:
    returns (dq, dk, dv, dq_weight, dk_weight), None for what is not there.  ``out``: the tensors to
    write the first three to (views of the qkv product's gradient, or the gradients that are given,
    as they lie).  The weights' gradients are summed in an order that the sizes fix, wherever the
    tensors lie."""
    parts, xs = (dq, dk, dv), (q, k)
    tokens, B, S, rot = _frequencies(dq, inv_freq, layout)
    out = _parts(parts, out, dq, tokens, rot)
    for i, (g, x) in enumerate(zip(parts, xs)):
        if (g is None) != (x is None):
            raise ValueError(f"{'qk'[i]} and its gradient go together")
        if g is not None:
            alike(x, "qk"[i], dq, g.shape)
            _heads(x, "qk"[i], dq, i, tokens, rot)
    wtype = _head_weights(q, k, dv, q_weight, k_weight)
    if q_weight is not None and k_weight is not None and q.shape[-1] != k.shape[-1]:
        raise ValueError("heads of q and k with weights must have one size")
    where, pos64, pb, pt = _positions(positions, start, dq, tokens, S)

    def launch(handle):
        res, packed, packed_x, weights, grads = [], [], [], [], []
        dws = [None if w is None else torch.empty_like(w) for w in (q_weight, k_weight)]
        for i, (t, o) in enumerate(zip(parts, out)):
            if t is None:
                res.append(None)
                continue
            res.append(_new(t) if o is None else o)
            if t.numel():
                packed.append(_pack(t, res[-1], i < 2))
                if i < 2:
                    packed_x.append(_pack(xs[i], xs[i], True))
                    weights.append((q_weight, k_weight)[i])
                    grads.append(dws[i])
            elif i < 2 and dws[i] is not None:
                dws[i].zero_()
        if weights:
            L = lib()
            D = max((g.numel() for g in grads if g is not None), default=0)
            ws = scratch(L.dash_rope_norm_bwd_workspace_bytes(D), q, workspace) if D else None
            none = [None] * (2 - len(weights))
            _check(L.dash_rope_norm_bwd(b"".join(packed), b"".join(packed_x), len(packed),
                                        _two(*weights, *none), _two(*grads, *none), B, S, rot,
                                        LAYOUTS[layout], DTYPES[dq.dtype], DTYPES[wtype],
                                        inv_freq.data_ptr(), magnitude, eps, where, pos64, pb, pt,
                                        start, None if ws is None else ws.data_ptr(),
                                        0 if ws is None else ws.numel() * ws.element_size(), handle),
                   "dash_rope_norm_bwd")
        elif packed:
            res[2].copy_(dv)
        return (*res, *dws)
    return run(dq, stream, launch)
