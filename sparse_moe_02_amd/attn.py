"""Query/key preparation with the append to a paged cache, and attention over that cache, on
device tensors (argument marshalling for ``include/attn.h``; every step runs in the HIP kernels).

Calls are enqueued on torch's current stream of the tensors' device and never wait for it.
"""

from __future__ import annotations

import torch

from . import binding as B
from ._device import N, on, stream

_DTYPES = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16}
_SCALINGS = {"none": B.MOE_ROPE_NONE, "linear": B.MOE_ROPE_LINEAR, "ntk": B.MOE_ROPE_NTK, "yarn": B.MOE_ROPE_YARN}


def rope_freqs(rot_dim: int, base: float = 1e4, scaling: str = "none", factor: float = 1.0, trained: int = 1,
               device=None):
    """Rotary frequencies (see ``moe_rope_freqs``): (float64 [rot_dim / 2] on device, mscale)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    f, mscale = B.moe_rope_freqs(rot_dim, base, _SCALINGS[scaling], factor, trained)
    return torch.tensor(f, dtype=torch.float64, device=device), mscale


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, inv_freq: torch.Tensor | None, *,
                mscale: float = 1.0, interleaved: bool = False, pos: torch.Tensor | None = None,
                row: torch.Tensor | None = None, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate the new tokens' queries and keys and append keys and values to the cache (see
    ``moe_rope_append``).

    q: [T][n_heads][D]; k, v: [T][n_kv_heads][D]; caches: [n_pages][page_size][n_kv_heads][D], any
    strides with a contiguous last dimension (slices of one projection, head-major pages, ...).
    table: int32 [n_rows][cols]; q_start: int32 [n_seqs + 1]; kv_len: int32 [n_rows], new tokens
    included; row: int32 [n_seqs] (default: sequence b has row b); pos: int32 [T] (default: each
    token's position); inv_freq: float64 [rot / 2] of ``rope_freqs`` (None: no rotation).  Returns
    q_out (may be q itself; by default a new tensor like q).  Tokens behind q_start[-1] are padding: their
    rows of q_out are left as they were (of a new tensor: unset)."""
    index = q.get_device()
    kv, n_kv, D, dtype = N.cache(k_cache, v_cache, index)
    b, _ = N.batch(table, q_start, kv_len, row, index)
    if q_out is None:
        q_out = torch.empty_like(q)
    hq, T, H = N.heads("q", q, -1, -1, D, dtype, index)
    ho = hq if q_out is q else N.heads("q_out", q_out, T, H, D, dtype, index)[0]
    hk = N.heads("k", k, T, n_kv, D, dtype, index)[0]
    hv = N.heads("v", v, T, n_kv, D, dtype, index)[0]
    fp, rot = None, 0
    if inv_freq is not None:
        fp, rot = N.address("inv_freq", inv_freq, N.FP64, index, -1), 2 * inv_freq.shape[0]
    pp = None if pos is None else N.address("pos", pos, N.INT32, index, T)
    if T:
        with on(index):
            st = (B._lib or B.lib()).moe_rope_append(kv, b, T, hq, ho, H, hk, hv, pp, fp, rot, mscale,
                                                     B.MOE_ROPE_INTERLEAVED if interleaved else 0, stream(index))
        if st:
            raise B.MoeError("moe_rope_append", st)
    return q_out


def paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
               q_start: torch.Tensor, kv_len: torch.Tensor, max_q: int, max_kv: int, *, scale: float | None = None,
               window: int = 0, full: bool = False, row: torch.Tensor | None = None, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None):
    """Attention of the new tokens over the paged cache (see ``moe_paged_attn``).

    Arguments as ``rope_append``; max_q and max_kv bound the new tokens and lengths (they shape the
    launch); scale defaults to head_dim ** -0.5; full: every token sees its whole sequence;
    window: only the last `window` positions.  workspace: uint8 tensor of
    ``paged_attn_workspace`` bytes (by default one is allocated for the call).  Returns out, or
    (out, lse) with lse float32 [T][n_heads] where lse is given or return_lse is set.  Rows of
    padding tokens behind q_start[-1] are left as they were (of a new tensor: unset)."""
    index = q.get_device()
    kv, _, D, dtype = N.cache(k_cache, v_cache, index)
    b, n_seqs = N.batch(table, q_start, kv_len, row, index)
    hq, T, H = N.heads("q", q, -1, -1, D, dtype, index)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    ho = N.heads("out", out, T, H, D, dtype, index)[0]
    lp = None if lse is None else N.address("lse", lse, N.FP32, index, T, H)
    if workspace is None:
        n = B.moe_paged_attn_workspace(kv, T, n_seqs, max_q, max_kv, H, window)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    wp, wn = None, 0
    if workspace is not None:
        wp, wn = N.address("workspace", workspace, N.UINT8, index), workspace.numel()
    if T:
        with on(index):
            st = (B._lib or B.lib()).moe_paged_attn(kv, b, T, max_q, max_kv, hq, H, ho, lp,
                                                    D ** -0.5 if scale is None else scale, window,
                                                    B.MOE_ATTN_FULL if full else 0, wp, wn, stream(index))
        if st:
            raise B.MoeError("moe_paged_attn", st)
    return out if lse is None else (out, lse)


def paged_attn_workspace(T: int, n_seqs: int, max_q: int, max_kv: int, n_heads: int, n_kv_heads: int, head_dim: int,
                         dtype: torch.dtype = torch.bfloat16, window: int = 0) -> int:
    """Bytes of workspace that ``paged_attn`` needs for these sizes."""
    kv = B.moe_paged_kv(None, None, 0, 0, 0, 1, 16, n_kv_heads, head_dim, _DTYPES[dtype])
    return B.moe_paged_attn_workspace(kv, T, n_seqs, max_q, max_kv, n_heads, window)
