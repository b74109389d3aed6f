"""Choice of tokens from logits, with the random numbers given, on device tensors (argument marshalling
for ``include/sample.h``; every step runs in the HIP kernels).

Calls are enqueued on torch's current stream of the logits' device and never wait for it.
"""

from __future__ import annotations

import torch

from . import binding as B
from ._device import N, on, stream

_TYPES = {torch.float32: B.MOE_FP32, torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16}


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
           top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None, *,
           out: torch.Tensor | None = None, prob: torch.Tensor | None = None, return_prob: bool = False,
           workspace: torch.Tensor | None = None):
    """A token for each row of logits (see ``moe_sample``).

    logits: [R][V], rows any distance apart, float32, bfloat16 or float16; u: float32 [R] in [0, 1);
    temperature (0: the largest logit), top_p, min_p: float32 [R], top_k: int32 [R], each None where it is
    off for all rows.  workspace: uint8 tensor of ``sample_workspace`` bytes (by default one is
    allocated for the call).  Returns int32 [R], or (tokens, probabilities) where prob is given or
    return_prob is set."""
    index = logits.get_device()
    t = _TYPES.get(logits.dtype)
    if t is None:
        raise ValueError("logits: float32, bfloat16 or float16 required")
    _, R, _, V = N.rows("logits", logits, -1, 1, -1, (N.BF16, N.FP16, N.FP32)[t], index)
    at, f32 = N.address, N.FP32
    up = at("u", u, f32, index, R)
    tp = None if temperature is None else at("temperature", temperature, f32, index, R)
    kp = None if top_k is None else at("top_k", top_k, N.INT32, index, R)
    pp = None if top_p is None else at("top_p", top_p, f32, index, R)
    mp = None if min_p is None else at("min_p", min_p, f32, index, R)
    if out is None:
        out = torch.empty_like(u, dtype=torch.int32)
    if prob is None and return_prob:
        prob = torch.empty_like(u)
    op = at("out", out, N.INT32, index, R)
    qp = None if prob is None else at("prob", prob, f32, index, R)
    if R:
        if workspace is None:
            workspace = torch.empty(B.moe_sample_workspace(R, V), dtype=torch.uint8, device=logits.device)
        wp = at("workspace", workspace, N.UINT8, index)
        with on(index):
            st = (B._lib or B.lib()).moe_sample(R, V, logits.data_ptr(), logits.stride(0) if R > 1 else 0, t, up, tp, kp, pp, mp,
                                                op, qp, wp, workspace.numel(), stream(index))
        if st:
            raise B.MoeError("moe_sample", st)
    return out if prob is None else (out, prob)


def sample_workspace(R: int, V: int) -> int:
    """Bytes of workspace that ``sample`` needs for R rows of V logits."""
    return B.moe_sample_workspace(R, V)
