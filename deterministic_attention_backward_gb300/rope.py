"""Rotary positions for the heads of a qkv product, forward and backward.

    inv_freq, magnitude = rope_freqs(128, base=10000.0)
    q, k, v = rope_fwd(q, k, v, inv_freq=inv_freq)          # turned, contiguous; v copied
    rope_bwd(dq, dk, dv, inv_freq=inv_freq, out=views_of_dqkv)

Heads are [B, S, H, D] (or packed [T, H, D]); any strides with contiguous heads, bf16, fp16 or
fp32.  One kernel launch turns q and k and copies v.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, lib
from ._args import DTYPES, disjoint, placed, shaped, tensor

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = ("none", "linear", "base", "ramp")


class _Part(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("D", ctypes.c_int), ("turn", ctypes.c_int), ("in_stride", ctypes.c_longlong * 3),
                ("out_stride", ctypes.c_longlong * 3)]


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
      index between; magnitude 0.1 ln(factor) + 1
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
        if original_len <= 0 or not fast > slow:
            raise ValueError("ramp wants original_len > 0 and fast > slow")
        turns = f * original_len / (2.0 * math.pi)
        first = float((turns > fast).sum())
        last = max(first + 1.0, float((turns > slow).sum()))
        p = torch.arange(rot // 2, dtype=torch.float64)
        keep = 1.0 - ((p - first) / (last - first)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0
    return f.to(device), magnitude


def _rope(parts, inv_freq, magnitude, positions, start, layout, out, stream, back):
    q = parts[0]
    tensor(q, "q", dtypes=DTYPES)
    if q.dim() not in (3, 4):
        raise ValueError(f"heads are [B, S, H, D] or [T, H, D], got {tuple(q.shape)}")
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    tensor(inv_freq, "inv_freq", dtypes=(torch.float64,))
    if inv_freq.device != q.device or inv_freq.dim() != 1 or not inv_freq.is_contiguous() or \
            not 0 < 2 * inv_freq.numel() <= 1024:
        raise ValueError("inv_freq must be contiguous float64 [rot/2] on the heads' device, "
                         "rot <= 1024")
    rot = 2 * inv_freq.numel()
    packed = q.dim() == 3
    B, S = (1, q.shape[0]) if packed else q.shape[:2]
    if out is not None and len(out) != len(parts):
        raise ValueError(f"out must hold {len(parts)} tensors")
    for i, t in enumerate(parts):
        name = "qkv"[i]
        if t is None:
            continue
        tensor(t, name, like=q)
        if t.shape[:-2] != q.shape[:-2] or t.dim() != q.dim():
            raise ValueError(f"{name} {tuple(t.shape)} does not go with q {tuple(q.shape)}")
        if i < 2 and t.shape[-1] < rot:
            raise ValueError(f"{name} has heads of {t.shape[-1]}, fewer than the {rot} that turn")
        for u, n in ((t, name), (out[i] if out is not None else None, f"out[{i}]")):
            if u is None:
                continue
            tensor(u, n, like=q)
            shaped(u, n, t.shape)
            if u.shape[-1] > 1 and u.stride(-1) != 1:
                raise ValueError(f"the elements of a head of {n} must be contiguous")
        if out is not None and out[i] is not None and not disjoint(out[i]):
            raise ValueError(f"out[{i}] has elements that share an address")
    pb = pt = 0
    if positions is not None:
        tensor(positions, "positions", dtypes=(torch.int32, torch.int64))
        if positions.device != q.device:
            raise ValueError(f"positions are on {positions.device}, the heads on {q.device}")
        want = (q.shape[0],) if packed else (B, S)
        if tuple(positions.shape) not in (want, want[-1:]):
            raise ValueError(f"positions must be {want} or {want[-1:]}, got "
                             f"{tuple(positions.shape)}")
        pt = positions.stride(-1)
        pb = positions.stride(0) if positions.dim() == 2 else 0
    with placed(q, stream):
        res = tuple(None if t is None else
                    out[i] if out is not None and out[i] is not None else
                    torch.empty(t.shape, dtype=t.dtype, device=t.device)
                    for i, t in enumerate(parts))
        arr, n = (_Part * 3)(), 0
        for i, (t, r) in enumerate(zip(parts, res)):
            if t is None or t.shape[-1] == 0 or t.shape[-2] == 0:
                continue
            a = arr[n]
            n += 1
            a.inp, a.out = t.data_ptr(), r.data_ptr()
            a.heads, a.D, a.turn = t.shape[-2], t.shape[-1], int(i < 2)
            a.in_stride[:] = (0, *t.stride()[:2]) if packed else t.stride()[:3]
            a.out_stride[:] = (0, *r.stride()[:2]) if packed else r.stride()[:3]
        if n and B and S:
            code = lib().dash_rope(arr, n, B, S, rot, LAYOUTS[layout], DTYPES[q.dtype],
                                   inv_freq.data_ptr(), float(magnitude),
                                   None if positions is None else positions.data_ptr(),
                                   int(positions is not None and positions.dtype == torch.int64),
                                   pb, pt, int(start), int(back),
                                   torch.cuda.current_stream().cuda_stream)
            _check(code, "dash_rope")
    return res


def rope_fwd(q, k=None, v=None, *, inv_freq, magnitude: float = 1.0, positions=None,
             start: int = 0, layout: str = "half", out=None, stream=None):
    """Turn the heads of q (and k) with their tokens' positions and copy v: returns (q, k, v),
    contiguous unless ``out`` gives the tensors to write (strided ones too; an input itself is
    turned in place).  Position of token s: ``positions`` (int32 or int64, [B, S] or [S];
    [T] for packed heads), or ``start`` + s."""
    return _rope((q, k, v), inv_freq, magnitude, positions, start, layout, out, stream, False)


def rope_bwd(dq, dk=None, dv=None, *, inv_freq, magnitude: float = 1.0, positions=None,
             start: int = 0, layout: str = "half", out=None, stream=None):
    """Gradient of ``rope_fwd``: from the gradients of its outputs those of its inputs
    (``out``: for example views of the qkv product's gradient)."""
    return _rope((dq, dk, dv), inv_freq, magnitude, positions, start, layout, out, stream, True)
