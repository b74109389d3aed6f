"""Root-mean-square norm with the residual's addition, and an output in 8 bits, on device tensors
(argument marshalling for ``include/norm.h``; every step runs in the HIP kernels).

Calls are enqueued on torch's current stream of the tensors' device and never wait for it.
"""

from __future__ import annotations

import torch

from . import binding as B
from ._device import N, on, stream

_TYPES = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16, torch.int8: B.MOE_INT8, torch.float8_e4m3fn: B.MOE_FP8}


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None, eps: float = 1e-6, *, offset: float = 0.0,
             residual: torch.Tensor | None = None, sum: torch.Tensor | None = None, out: torch.Tensor | None = None,
             out_dtype: torch.dtype | None = None, group: int = 0, scale: torch.Tensor | None = None):
    """h = x + residual, y = h * (mean(h^2) + eps)^(-1/2) * (offset + weight) (see ``moe_rms_norm``).

    x, residual: bfloat16 or float16 [T][D] or [T][n][D] (rows normalised one by one), any strides with
    a contiguous last dimension; weight: [D] of the same type.  out_dtype: x's type (the default),
    torch.int8 or torch.float8_e4m3fn; then y is codes * scale, with a scale for each row or, where
    group is 32, 64 or 128, for each group elements of it: float32 [T](x[n])[1 or D / group].
    sum takes h (may be x or residual itself; by default a new tensor where there is a residual);
    out, of x's type, may be x or residual itself.

    Returns y; (y, h) with a residual or sum; (codes, scale) or (codes, scale, h) in 8 bits."""
    index = x.get_device()
    type_ = x.dtype
    if type_ not in (torch.bfloat16, torch.float16):
        raise ValueError("x: bfloat16 or float16 required")
    kind = N.BF16 if type_ is torch.bfloat16 else N.FP16
    hx, T, n, D = N.rows("x", x, -1, -1, -1, kind, index)
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = type_
    codes = out_dtype is not type_
    if codes and out_dtype not in (torch.int8, torch.float8_e4m3fn):
        raise ValueError("out_dtype: x's type, torch.int8 or torch.float8_e4m3fn required")
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype, memory_format=torch.contiguous_format)
    if sum is None and residual is not None:
        sum = torch.empty_like(x, memory_format=torch.contiguous_format)
    if codes:
        groups = D // group if group > 0 and D > 0 else 1
        if scale is None:
            scale = torch.empty((*x.shape[:-1], groups), dtype=torch.float32, device=x.device)
        sp = N.address("scale", scale, N.FP32, index, *x.shape[:-1], groups)
    else:
        if scale is not None:
            raise ValueError("scale: for outputs in 8 bits only")
        sp = None
    ho = N.rows("out", out, T, n, D, (N.INT8 if out_dtype is torch.int8 else N.FP8) if codes else kind, index)[0]
    hr = None if residual is None else N.rows("residual", residual, T, n, D, kind, index)[0]
    hs = None if sum is None else N.rows("sum", sum, T, n, D, kind, index)[0]
    wp = None if weight is None else N.address("weight", weight, kind, index, D)
    if T * n * D:
        with on(index):
            st = (B._lib or B.lib()).moe_rms_norm(T, n, D, _TYPES[type_], hx, hr, hs, wp, offset, eps, _TYPES[out_dtype], ho,
                                                  group, sp, stream(index))
        if st:
            raise B.MoeError("moe_rms_norm", st)
    if codes:
        return (out, scale) if sum is None else (out, scale, sum)
    return out if sum is None else (out, sum)
