"""Rotary positions for the heads of a qkv product, forward and backward.

    inv_freq, magnitude = rope_freqs(128, base=10000.0)
    q, k, v = rope_fwd(q, k, v, inv_freq=inv_freq)          # turned, contiguous; v copied
    rope_bwd(dq, dk, dv, inv_freq=inv_freq, out=views_of_dqkv)

Heads are [B, S, H, D] (or packed [T, H, D]); any strides with contiguous heads, bf16, fp16 or
fp32.  One kernel launch turns q and k and copies v.
"""
from __future__ import annotations

import math
import struct

import torch

from . import _check, lib
from ._args import DTYPES, alike, disjoint, run, tensor

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


def _rope(parts, inv_freq, magnitude, positions, start, layout, out, stream, back):
    q = parts[0]
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
    given = out is not None
    out = tuple(out) if given else (None, None, None)
    if len(out) != len(parts):
        raise ValueError(f"out must hold {len(parts)} tensors")
    res, packed = [], []
    for i, t in enumerate(parts):
        if t is None:
            continue
        name, shape = "qkv"[i], t.shape
        if i:
            alike(t, name, q)
            if shape[:-2] != tokens or t.dim() != dims:
                raise ValueError(f"{name} {tuple(shape)} does not go with q {tuple(q.shape)}")
        if i < 2 and shape[-1] < rot:
            raise ValueError(f"{name} has heads of {shape[-1]}, fewer than the {rot} that turn")
        if shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"the elements of a head of {name} must be contiguous")
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
    where, pos64, pb, pt = None, 0, 0, 0
    if positions is None:
        if not -2 ** 63 <= start <= 2 ** 63 - S:
            raise ValueError(f"positions from {start} on do not fit 64 bits")
    else:
        tensor(positions, "positions", (torch.int32, torch.int64))
        if positions.device != q.device:
            raise ValueError(f"positions are on {positions.device}, the heads on {q.device}")
        if positions.shape != tokens and positions.shape != tokens[-1:]:
            raise ValueError(f"positions must be {tuple(tokens)} or {tuple(tokens[-1:])}, got "
                             f"{tuple(positions.shape)}")
        where, pos64 = positions.data_ptr(), int(positions.dtype == torch.int64)
        pt = positions.stride(-1)
        pb = positions.stride(0) if positions.dim() == 2 else 0

    def launch(handle):
        for t, o in zip(parts, out):
            if t is None:
                res.append(None)
                continue
            if o is None:
                o = torch.empty_like(t) if t.is_contiguous() else \
                    torch.empty(t.shape, dtype=t.dtype, device=t.device)
            res.append(o)
            if t.numel():
                ti, to = t.stride(), o.stride()
                if dims == 3:
                    ti, to = (0, *ti), (0, *to)
                packed.append(_PART.pack(t.data_ptr(), o.data_ptr(), t.shape[-2], t.shape[-1],
                                         int(len(res) < 3), ti[0], ti[1], ti[2], to[0], to[1],
                                         to[2]))
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
