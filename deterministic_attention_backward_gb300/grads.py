"""The norm over many gradients, and clipping by it.

    norm = grad_norm(grads)                         # fp32 scalar on the device, nothing waits for it
    norm = grad_clip(grads, max_norm=1.0)           # in place: g *= min(1, max_norm / (norm + eps))
    norm = grad_clip(grads, max_norm=1.0, out=buffers)

``grads`` are tensors of one device, bf16, fp16 and fp32 mixed, of any sizes (None is passed over), each
dense in memory in some order of its dimensions.  Sums run in an order that the sizes fix: the same
bits on every run, wherever the tensors lie.
"""
from __future__ import annotations

import struct

import torch

from . import _check, lib
from ._args import DTYPES, Tensor, alike, disjoint, run, scratch, tensor

_GRAD = struct.Struct("@PPqii")  # dash_grad_t: in, out, n, dtype, -


def _dense(t):
    """Whether the elements of ``t`` lie next to each other, in some order."""
    if t.is_contiguous() or t.numel() == 0:
        return True
    return sum((n - 1) * s for n, s in zip(t.shape, t.stride())) == t.numel() - 1 and disjoint(t)


def _list(grads, name="grads"):
    """The gradients that are there, checked."""
    if isinstance(grads, Tensor):
        grads = (grads,)
    grads = [t for t in grads if t is not None]
    if not grads:
        raise ValueError(f"{name} holds no tensor")
    tensor(grads[0], f"{name}[0]", DTYPES)
    device = grads[0].get_device()
    for i, t in enumerate(grads):
        if not isinstance(t, Tensor) or t.get_device() != device or t.dtype not in DTYPES:
            tensor(t, f"{name}[{i}]", DTYPES)
            raise ValueError(f"{name}[{i}] is on {t.device}, expected {grads[0].device}")
        if not t.is_contiguous() and not _dense(t):
            raise ValueError(f"{name}[{i}] must be dense in memory, got strides {tuple(t.stride())}")
    return grads


def _pack(grads, outs=None):
    """The tensors as an array of dash_grad_t."""
    if outs is None:
        rows = [(p, p, t.numel(), DTYPES[t.dtype], 0) for t in grads for p in (t.data_ptr(),)]
    else:
        rows = [(t.data_ptr(), o.data_ptr(), t.numel(), DTYPES[t.dtype], 0)
                for t, o in zip(grads, outs)]
    return b"".join([_GRAD.pack(*r) for r in rows])


def _scalar(t, name, like):
    alike(t, name, like, dtype=torch.float32)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value, got {tuple(t.shape)}")


def grad_norm_workspace_bytes(count: int) -> int:
    """Workspace bytes of ``grad_norm`` and ``grad_clip`` for ``count`` tensors."""
    return int(lib().dash_grad_norm_workspace_bytes(count))


def grad_norm(grads, *, out=None, workspace=None, stream=None):
    """The square root of the sum of squares over all tensors: an fp32 scalar on their device
    (``out`` where one is given)."""
    grads = _list(grads)
    like = grads[0]
    if out is not None:
        _scalar(out, "out", like)

    def launch(handle):
        L, n = lib(), len(grads)
        norm = torch.empty((), dtype=torch.float32, device=like.device) if out is None else out
        ws = scratch(L.dash_grad_norm_workspace_bytes(n), like, workspace)
        _check(L.dash_grad_norm(_pack(grads), n, norm.data_ptr(), ws.data_ptr(),
                                ws.numel() * ws.element_size(), handle), "dash_grad_norm")
        return norm
    return run(like, stream, launch)


def grad_clip(grads, max_norm: float, *, eps: float = 1e-6, norm=None, out=None, workspace=None,
              stream=None):
    """Scale the gradients by min(1, max_norm / (norm + eps)), in place or into the tensors ``out``
    (one for each gradient, like it), and return the norm they had.  ``norm``: one that is known
    already, for example over more tensors than these.  Within the limit nothing is written in place.
    A norm that is NaN makes every gradient NaN; one that is infinite makes the finite ones zero.  An
    infinite ``max_norm`` clips nothing, whatever the norm's value."""
    grads = _list(grads)
    like = grads[0]
    if not max_norm >= 0 or not eps >= 0:
        raise ValueError(f"max_norm and eps must not be negative, got {max_norm} and {eps}")
    if norm is not None:
        _scalar(norm, "norm", like)
    outs = None
    if out is not None:
        outs = [o for o in ((out,) if isinstance(out, Tensor) else out) if o is not None]
        if len(outs) != len(grads):
            raise ValueError(f"out must hold {len(grads)} tensors, got {len(outs)}")
        for i, (t, o) in enumerate(zip(grads, outs)):
            alike(o, f"out[{i}]", t, t.shape)
            if o.stride() != t.stride() and not (o.is_contiguous() and t.is_contiguous()):
                raise ValueError(f"out[{i}] must have strides {tuple(t.stride())}, got "
                                 f"{tuple(o.stride())}")

    def launch(handle):
        L, n = lib(), len(grads)
        res = torch.empty((), dtype=torch.float32, device=like.device) if norm is None else norm
        ws = scratch(L.dash_grad_norm_workspace_bytes(n), like, workspace) if norm is None else None
        _check(L.dash_grad_clip(_pack(grads, outs), n, max_norm, eps,
                                None if norm is None else norm.data_ptr(),
                                res.data_ptr() if norm is None else None,
                                None if ws is None else ws.data_ptr(),
                                0 if ws is None else ws.numel() * ws.element_size(), handle),
               "dash_grad_clip")
        return res
    return run(like, stream, launch)
