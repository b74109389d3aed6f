"""What the wrappers ask torch for on every call, kept short: a small call's time is the host's."""

from __future__ import annotations

import contextlib

import torch

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_here = contextlib.nullcontext()


def stream(index: int) -> int:
    """hipStream_t of torch's current stream on a device."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def on(index: int):
    """Context in which the device is the current one."""
    return _here if torch.cuda.current_device() == index else torch.cuda.device(index)


def int32(name: str, t: torch.Tensor, index: int) -> int:
    """Address of a contiguous int32 tensor on the device."""
    if t.dtype is not torch.int32 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous torch.int32 tensor on cuda:{index} required")
    return t.data_ptr()
