"""Argument checks and placement shared by the operators around the attention."""
from __future__ import annotations

import contextlib

import torch

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def tensor(t, name, like=None, dtypes=None):
    """Raise ValueError unless ``t`` is a CUDA tensor (on ``like``'s device and of its type) of
    one of ``dtypes``."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if dtypes is None and like is not None and t.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype}, got {t.dtype}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")


def shaped(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def disjoint(t) -> bool:
    """Whether no two elements of ``t`` share an address (it can be written)."""
    reach = 0
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size > 1:
            if stride <= reach:
                return False
            reach += stride * (size - 1)
    return True


_here = contextlib.nullcontext()


def placed(t, stream):
    """Context in which a call on ``t`` allocates and launches: ``stream`` where one is given
    (its own memory pool, so that temporaries are reused in its order only), otherwise the
    current stream of ``t``'s device."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.device.index != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return _here
