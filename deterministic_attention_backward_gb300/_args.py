"""Argument checks and placement shared by the operators around the attention.

The checks run on every call, and a call on a few rows takes less time on the GPU than they do,
so each looks at a tensor once and takes the short way where it is contiguous.
"""
from __future__ import annotations

import torch

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
Tensor = torch.Tensor

# the current stream's handle by device index, without building a Stream object
try:
    raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def tensor(t, name, dtypes):
    """Raise ValueError unless ``t`` is a CUDA tensor of one of ``dtypes``."""
    if not isinstance(t, Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")


def alike(t, name, like, shape=None, dtype=None):
    """Raise ValueError unless ``t`` is a tensor on ``like``'s device, of its type (or ``dtype``)
    and, where one is given, of ``shape``."""
    if not isinstance(t, Tensor):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.dtype != (dtype or like.dtype):
        raise ValueError(f"{name} must be {dtype or like.dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def contiguous(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def apart(outs, others=()):
    """Raise ValueError where two of the tensors ``outs`` that a call writes begin at one address,
    or one of them where one of ``others`` does that it reads."""
    at = [t.data_ptr() for t in outs if t is not None and t.numel()]
    if len(set(at)) < len(at):
        raise ValueError("two outputs are the same memory")
    if not set(at).isdisjoint(t.data_ptr() for t in others if t is not None):
        raise ValueError("an output is the memory of an input")


def scratch(nbytes, like, given):
    """A workspace on ``like``'s device: ``given``, checked, or a new one."""
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    if not isinstance(given, Tensor) or given.device != like.device:
        raise ValueError(f"workspace must be a tensor on {like.device}")
    contiguous(given, "workspace")
    if given.numel() * given.element_size() < nbytes:
        raise ValueError(f"workspace too small: {nbytes} bytes are needed")
    return given


def disjoint(t) -> bool:
    """Whether no two elements of ``t`` share an address (it can be written)."""
    if t.is_contiguous():
        return True
    reach = 0
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size > 1:
            if stride <= reach:
                return False
            reach += stride * (size - 1)
    return True


def placed(t, stream):
    """Context in which a call on ``t`` allocates and launches: ``stream`` where one is given
    (its own memory pool, so that temporaries are reused in its order only), otherwise the
    current stream of ``t``'s device; None where that is current already."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return None


def run(t, stream, launch):
    """``launch(stream handle)`` in the context of ``placed``."""
    ctx = placed(t, stream)
    if ctx is None:
        return launch(raw_stream(t.get_device()))
    with ctx:
        return launch(raw_stream(t.get_device()))
