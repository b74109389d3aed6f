"""What the wrappers ask torch for on every call, kept short: a small call's time is the host's."""

from __future__ import annotations

import contextlib

import torch


class _NotBuilt:
    """In the tensor reader's place where it has not been built: its first use says so (or finds
    it, if it was built since), so that what needs the library alone can be imported and run."""

    def __getattr__(self, name):
        try:
            from . import _tensors
        except ImportError as e:
            raise ImportError(f"the tensor reader is not built ({e}): run __graft_entry__.build()") from e
        return getattr(_tensors, name)


try:
    from . import _tensors as N  # noqa: F401
except ImportError:  # built with the library
    N = _NotBuilt()

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_here = contextlib.nullcontext()


def stream(index: int) -> int:
    """hipStream_t of torch's current stream on a device."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def on(index: int):
    """Context in which the device is the current one."""
    return _here if _device() == index else torch.cuda.device(index)
