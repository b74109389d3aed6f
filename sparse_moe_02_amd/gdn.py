"""Gated DeltaNet prefill scan and decode step on device tensors (argument marshalling for
``moe_gdn_scan`` and ``moe_gdn_step`` of ``include/gdn.h``; every step runs in the HIP kernels)."""

from __future__ import annotations

import torch

from . import binding as B
from ._device import N, on, stream

D = 128


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def gdn_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
             state: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scan T tokens.  q, k: bf16 [T][n_kheads][128]; v: bf16 [T][n_vheads][128]; alpha, beta:
    float32 [T][n_vheads]; state: float32 [n_vheads][128][128], updated in place.
    Returns out (bf16 [T][n_vheads][128])."""
    T, hk, dk = k.shape
    hv, dv = v.shape[1], v.shape[2]
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("alpha", alpha, torch.float32), ("beta", beta, torch.float32),
                        ("state", state, torch.float32)):
        if t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous {dt} device tensor required")
    if q.shape != k.shape or v.shape[0] != T or alpha.shape != (T, hv) or beta.shape != (T, hv):
        raise ValueError("shape mismatch")
    if state.shape != (hv, dv, dk):
        raise ValueError("state must be [n_vheads][d_v][d_k]")
    if out is None:
        out = torch.empty((T, hv, dv), dtype=torch.bfloat16, device=v.device)
    s = stream if stream is not None else torch.cuda.current_stream(v.device).cuda_stream
    B.moe_gdn_scan(T, hk, hv, dk, dv, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(out),
                   s)
    return out


def gdn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
             state: torch.Tensor, slot: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """One token each of R rows; row r updates state slot[r] in place, rows of one slot in row
    order (see ``moe_gdn_step``).  q, k: bf16 [R][n_kheads][128]; v: bf16 [R][n_vheads][128];
    alpha, beta: float32 [R][n_vheads]; state: float32 [n_slots][n_vheads][128][128]; slot: int32
    [R] (outside the pool: padding, zeros out).  Returns out (bf16 [R][n_vheads][128]); enqueued on
    torch's current stream of the tensors' device."""
    if k.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q, k, v must be [R][heads][128] and state [n_slots][n_vheads][128][128]")
    R, hk, dk = k.shape
    _, hv, dv = v.shape
    index, n_slots = v.get_device(), state.shape[0]
    if out is None:
        out = torch.empty_like(v)
    at, bf16, f32 = N.address, N.BF16, N.FP32
    args = (at("q", q, bf16, index, R, hk, dk), at("k", k, bf16, index, R, hk, dk), at("v", v, bf16, index, R, hv, dv),
            at("alpha", alpha, f32, index, R, hv), at("beta", beta, f32, index, R, hv),
            at("state", state, f32, index, n_slots, hv, dv, dk), n_slots, at("slot", slot, N.INT32, index, R),
            at("out", out, bf16, index, R, hv, dv))
    with on(index):
        st = (B._lib or B.lib()).moe_gdn_step(R, hk, hv, dk, dv, *args, stream(index))
    if st:
        raise B.MoeError("moe_gdn_step", st)
    return out
