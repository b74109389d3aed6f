"""Query/key preparation with the append to a paged cache, and attention over that cache, on
device tensors (argument marshalling for ``include/attn.h``; every step runs in the HIP kernels).

Calls are enqueued on torch's current stream of the tensors' device and never wait for it.
"""

from __future__ import annotations

import torch

from . import binding as B

_DTYPES = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16}
_SCALINGS = {"none": B.MOE_ROPE_NONE, "linear": B.MOE_ROPE_LINEAR, "ntk": B.MOE_ROPE_NTK, "yarn": B.MOE_ROPE_YARN}


def rope_freqs(rot_dim: int, base: float = 1e4, scaling: str = "none", factor: float = 1.0, trained: int = 1,
               device=None):
    """Rotary frequencies (see ``moe_rope_freqs``): (float64 [rot_dim / 2] on device, mscale)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    f, mscale = B.moe_rope_freqs(rot_dim, base, _SCALINGS[scaling], factor, trained)
    return torch.tensor(f, dtype=torch.float64, device=device), mscale


def _need(name, t, dtype, device, dim=None):
    if t.dtype != dtype or t.device != device or (dim is not None and t.dim() != dim):
        raise ValueError(f"{name}: {dtype} tensor{'' if dim is None else f' of {dim} dimensions'} on {device} required")


def _ints(name, t, device, dim):
    _need(name, t, torch.int32, device, dim)
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor required")
    return t.data_ptr()


def _heads(name, t, T, heads, D, dtype, device):
    _need(name, t, dtype, device, 3)
    if t.shape != (T, heads, D) or (D > 1 and t.stride(2) != 1):
        raise ValueError(f"{name}: [{T}][{heads}][{D}] with a contiguous last dimension required")
    # strides of dimensions of one element say nothing
    return B.moe_heads(t.data_ptr(), t.stride(0) if T > 1 else 0, t.stride(1) if heads > 1 else 0)


def _cache(k_cache, v_cache, device):
    if k_cache.dtype not in _DTYPES or not k_cache.is_cuda or k_cache.device != device or k_cache.dim() != 4:
        raise ValueError(f"k_cache: bfloat16 or float16 [n_pages][page_size][n_kv_heads][head_dim] on {device} required")
    if v_cache.dtype != k_cache.dtype or v_cache.device != device or v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must have k_cache's type, device and shape")
    n_pages, page, heads, D = k_cache.shape
    st = [s if n > 1 else 0 for s, n in zip(k_cache.stride(), k_cache.shape)]
    if st != [s if n > 1 else 0 for s, n in zip(v_cache.stride(), v_cache.shape)] or st[3] != 1:
        raise ValueError("k_cache and v_cache must have the same strides and a contiguous last dimension")
    return B.moe_paged_kv(k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], n_pages, page, heads, D,
                          _DTYPES[k_cache.dtype])


def _batch(table, q_start, kv_len, row, device):
    n = q_start.shape[0] - 1 if q_start.dim() == 1 else -1
    if row is not None and (row.dim() != 1 or row.shape[0] != n):
        raise ValueError("row: int32 [n_seqs] required")
    b = B.moe_batch(_ints("q_start", q_start, device, 1), _ints("kv_len", kv_len, device, 1),
                    _ints("table", table, device, 2), None if row is None else _ints("row", row, device, 1), n,
                    table.shape[0], table.shape[1])
    if kv_len.shape[0] != table.shape[0]:
        raise ValueError("kv_len must have one entry for each row of table")
    return b


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
    q_out (may be q itself; by default a new tensor).  Tokens behind q_start[-1] are padding: their
    rows of q_out are left as they were (of a new tensor: unset)."""
    dev = q.device
    kv = _cache(k_cache, v_cache, dev)
    b = _batch(table, q_start, kv_len, row, dev)
    if q.dim() != 3:
        raise ValueError("q: [T][n_heads][head_dim] required")
    T, H, D = q.shape[0], q.shape[1], kv.head_dim
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    hq = _heads("q", q, T, H, D, k_cache.dtype, dev)
    ho = _heads("q_out", q_out, T, H, D, k_cache.dtype, dev)
    hk = _heads("k", k, T, kv.n_kv_heads, D, k_cache.dtype, dev)
    hv = _heads("v", v, T, kv.n_kv_heads, D, k_cache.dtype, dev)
    fp, rot = None, 0
    if inv_freq is not None:
        _need("inv_freq", inv_freq, torch.float64, dev, 1)
        if not inv_freq.is_contiguous():
            raise ValueError("inv_freq: contiguous tensor required")
        fp, rot = inv_freq.data_ptr(), 2 * inv_freq.shape[0]
    pp = None
    if pos is not None:
        pp = _ints("pos", pos, dev, 1)
        if pos.shape[0] != T:
            raise ValueError("pos: int32 [T] required")
    if T == 0:
        return q_out
    with torch.cuda.device(dev):
        B.moe_rope_append(kv, b, T, hq, ho, H, hk, hv, pp, fp, rot, mscale,
                          B.MOE_ROPE_INTERLEAVED if interleaved else 0, torch.cuda.current_stream(dev).cuda_stream)
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
    dev = q.device
    kv = _cache(k_cache, v_cache, dev)
    b = _batch(table, q_start, kv_len, row, dev)
    if q.dim() != 3:
        raise ValueError("q: [T][n_heads][head_dim] required")
    T, H, D = q.shape[0], q.shape[1], kv.head_dim
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    hq = _heads("q", q, T, H, D, k_cache.dtype, dev)
    ho = _heads("out", out, T, H, D, k_cache.dtype, dev)
    lp = None
    if lse is not None:
        _need("lse", lse, torch.float32, dev, 2)
        if lse.shape != (T, H) or not lse.is_contiguous():
            raise ValueError("lse: contiguous float32 [T][n_heads] required")
        lp = lse.data_ptr()
    n = B.moe_paged_attn_workspace(kv, T, b.n_seqs, max_q, max_kv, H, window)
    if workspace is None:
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        _need("workspace", workspace, torch.uint8, dev, 1)
        if not workspace.is_contiguous():
            raise ValueError("workspace: contiguous uint8 tensor required")
    wp, wn = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    if T:
        with torch.cuda.device(dev):
            B.moe_paged_attn(kv, b, T, max_q, max_kv, hq, H, ho, lp, D ** -0.5 if scale is None else scale, window,
                             B.MOE_ATTN_FULL if full else 0, wp, wn, torch.cuda.current_stream(dev).cuda_stream)
    return out if lse is None else (out, lse)


def paged_attn_workspace(T: int, n_seqs: int, max_q: int, max_kv: int, n_heads: int, n_kv_heads: int, head_dim: int,
                         dtype: torch.dtype = torch.bfloat16, window: int = 0) -> int:
    """Bytes of workspace that ``paged_attn`` needs for these sizes."""
    kv = B.moe_paged_kv(None, None, 0, 0, 0, 1, 16, n_kv_heads, head_dim, _DTYPES[dtype])
    return B.moe_paged_attn_workspace(kv, T, n_seqs, max_q, max_kv, n_heads, window)
