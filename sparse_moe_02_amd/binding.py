"""ctypes binding of ``include/moe.h`` -- argument marshalling only.

Every function keeps the C name and raises :class:`MoeError` on a non-OK status.
All computation happens in the HIP library (``libmoe_mi355x.so``); if it has not been
built, loading fails loudly -- there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

MOE_BF16, MOE_FP16, MOE_FP32, MOE_INT8, MOE_FP8 = range(5)
MOE_OK = 0
MOE_STAGE_ROUTE, MOE_STAGE_GROUP, MOE_STAGE_GATEUP, MOE_STAGE_DOWN, MOE_STAGE_FINAL = range(5)
MOE_PREFILL_STAGES = 5
MOE_DSTAGE_LAYER = 0
MOE_DECODE_STAGES = 1
PREFILL_STAGE_NAMES = ("route", "group", "gateup", "down", "final")
DECODE_STAGE_NAMES = ("layer",)
CTRL_DECODE_ERR_OFFSET = 88  # byte offset of the decode wait-failure word in the workspace

STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_DTYPE", 4: "MOE_ERR_ALIGN",
                5: "MOE_ERR_WORKSPACE", 6: "MOE_ERR_TOKENS", 7: "MOE_ERR_DEVICE", 8: "MOE_ERR_HIP",
                9: "MOE_ERR_ALIAS", 10: "MOE_ERR_ALLOC", 11: "MOE_ERR_WAIT"}
(MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_TOKENS, MOE_ERR_DEVICE,
 MOE_ERR_HIP, MOE_ERR_ALIAS, MOE_ERR_ALLOC, MOE_ERR_WAIT) = range(1, 12)
assert all(STATUS_NAMES[globals()[n] if n != "MOE_OK" else 0] == n for n in STATUS_NAMES.values())

# moe_config.flags (include/moe.h)
MOE_F_NONE = 0


def MOE_F_FORCE_BM(rows: int) -> int:
    return (rows // 32) & 0xF


MOE_F_NO_FALLBACK = 1 << 4
MOE_F_SEPARATE_DEQUANT = 1 << 5
MOE_F_HOST_ROUTING = 1 << 6

EXPORTED = ("moe_plan_create", "moe_plan_destroy", "moe_workspace_init", "moe_workspace_check",
            "moe_forward_prefill", "moe_forward_decode", "moe_forward_decode_batch", "moe_forward_decode_static",
            "moe_pack_qparams",
            "moe_pack_codes", "moe_status_string", "moe_version", "moe_gdn_scan", "moe_gdn_step", "moe_rope_freqs",
            "moe_rope_append", "moe_paged_attn_workspace", "moe_paged_attn", "moe_pages_workspace", "moe_pages_grow",
            "moe_pages_fork", "moe_pages_free", "moe_pages_compact", "moe_pages_copy", "moe_pages_check", "moe_rms_norm",
            "moe_linear", "moe_sample_workspace", "moe_sample", "moe_prefix_attn_workspace", "moe_prefix_attn")

# include/attn.h
MOE_ROPE_NONE, MOE_ROPE_LINEAR, MOE_ROPE_NTK, MOE_ROPE_YARN = range(4)
MOE_ROPE_INTERLEAVED = 1
MOE_ATTN_FULL = 1


class moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("group_size", ctypes.c_int32), ("router_dtype", ctypes.c_int),
                ("qparam_dtype", ctypes.c_int), ("max_chunk_tokens", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class moe_qmat(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class moe_weights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p), ("gate", moe_qmat),
                ("up", moe_qmat), ("down", moe_qmat), ("s_gate", moe_qmat), ("s_up", moe_qmat),
                ("s_down", moe_qmat), ("shared_gate", ctypes.c_void_p)]


class moe_debug_out(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("gates", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("row_token", ctypes.c_void_p), ("n_refined", ctypes.c_void_p),
                ("events", ctypes.c_void_p), ("logits32", ctypes.c_void_p), ("radii32", ctypes.c_void_p)]


class moe_heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class moe_paged_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int)]


class moe_batch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("row", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("table_cols", ctypes.c_int32)]


class moe_prefix_groups(ctypes.Structure):
    _fields_ = [("group_start", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p), ("n_groups", ctypes.c_int32)]


class moe_pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("len", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("table_cols", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class moe_page_memory(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("plane_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("page_bytes", ctypes.c_int64), ("n_planes", ctypes.c_int32)]


class moe_linear_weights(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("qparam_dtype", ctypes.c_int)]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                                   "(there is no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
            L.moe_plan_create.restype = ctypes.c_int
            L.moe_plan_create.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights),
                                          ctypes.POINTER(P), ctypes.POINTER(SZ)]
            L.moe_plan_destroy.restype = None
            L.moe_plan_destroy.argtypes = [P]
            L.moe_workspace_init.restype = ctypes.c_int
            L.moe_workspace_init.argtypes = [P, P, SZ, P]
            L.moe_workspace_check.restype = ctypes.c_int
            L.moe_workspace_check.argtypes = [P, P, SZ, P]
            L.moe_forward_prefill.restype = ctypes.c_int
            L.moe_forward_prefill.argtypes = [P, P, I64, P, P, SZ, P, ctypes.POINTER(moe_debug_out)]
            L.moe_forward_decode.restype = ctypes.c_int
            L.moe_forward_decode.argtypes = [P, P, P, P, SZ, P, ctypes.POINTER(moe_debug_out)]
            L.moe_forward_decode_batch.restype = ctypes.c_int
            L.moe_forward_decode_batch.argtypes = [P, P, ctypes.c_int32, P, P, SZ, P, ctypes.POINTER(moe_debug_out)]
            L.moe_forward_decode_static.restype = ctypes.c_int
            L.moe_forward_decode_static.argtypes = [P, P, P, P, ctypes.POINTER(moe_debug_out)]
            L.moe_pack_qparams.restype = ctypes.c_int
            L.moe_pack_qparams.argtypes = [P, P, I64, ctypes.c_int32, P]
            L.moe_pack_codes.restype = ctypes.c_int
            L.moe_pack_codes.argtypes = [P, P, I64, ctypes.c_int32, P]
            L.moe_gdn_scan.restype = ctypes.c_int
            L.moe_gdn_scan.argtypes = [ctypes.c_int32] * 5 + [P] * 7 + [P]
            L.moe_gdn_step.restype = ctypes.c_int
            L.moe_gdn_step.argtypes = [ctypes.c_int32] * 5 + [P] * 6 + [ctypes.c_int32, P, P, P]
            KV = BA = HD = P  # structures by reference, or their bytes (see _ref)
            L.moe_rope_freqs.restype = ctypes.c_int
            L.moe_rope_freqs.argtypes = [ctypes.c_int32, ctypes.c_double, ctypes.c_int, ctypes.c_double, I64, P, P]
            L.moe_rope_append.restype = ctypes.c_int
            L.moe_rope_append.argtypes = [KV, BA, I64, HD, HD, ctypes.c_int32, HD, HD, P, P, ctypes.c_int32,
                                          ctypes.c_float, ctypes.c_uint32, P]
            L.moe_paged_attn_workspace.restype = ctypes.c_int
            L.moe_paged_attn_workspace.argtypes = [KV, I64, ctypes.c_int32, I64, I64, ctypes.c_int32, ctypes.c_int32,
                                                   ctypes.POINTER(SZ)]
            L.moe_paged_attn.restype = ctypes.c_int
            L.moe_paged_attn.argtypes = [KV, BA, I64, I64, I64, HD, ctypes.c_int32, HD, P, ctypes.c_float,
                                         ctypes.c_int32, ctypes.c_uint32, P, SZ, P]
            PG = PM = P
            I32 = ctypes.c_int32
            L.moe_pages_workspace.restype = ctypes.c_int
            L.moe_pages_workspace.argtypes = [PG, I32, ctypes.POINTER(SZ)]
            L.moe_pages_grow.restype = ctypes.c_int
            L.moe_pages_grow.argtypes = [PG, PG, I32, P, P, P, P, SZ, P]
            L.moe_pages_fork.restype = ctypes.c_int
            L.moe_pages_fork.argtypes = [PG, PG, PM, I32, P, P, P, P, SZ, P]
            L.moe_pages_free.restype = ctypes.c_int
            L.moe_pages_free.argtypes = [PG, PG, I32, P, P, P, SZ, P]
            L.moe_pages_compact.restype = ctypes.c_int
            L.moe_pages_compact.argtypes = [PG, PG, PM, P, P, SZ, P]
            L.moe_pages_copy.restype = ctypes.c_int
            L.moe_pages_copy.argtypes = [PM, I32, I32, P, P, P]
            L.moe_pages_check.restype = ctypes.c_int
            L.moe_pages_check.argtypes = [P, P]
            F32 = ctypes.c_float
            L.moe_rms_norm.restype = ctypes.c_int
            L.moe_rms_norm.argtypes = [I64, I32, I32, ctypes.c_int, HD, HD, HD, P, F32, F32, ctypes.c_int, HD, I32, P, P]
            L.moe_linear.restype = ctypes.c_int
            L.moe_linear.argtypes = [P, I64, P, I64, ctypes.c_int, P, I32, P, I64, ctypes.c_int, P]
            L.moe_sample_workspace.restype = ctypes.c_int
            L.moe_sample_workspace.argtypes = [I64, I32, ctypes.POINTER(SZ)]
            L.moe_sample.restype = ctypes.c_int
            L.moe_sample.argtypes = [I64, I32, P, I64, ctypes.c_int, P, P, P, P, P, P, P, P, SZ, P]
            L.moe_prefix_attn_workspace.restype = ctypes.c_int
            L.moe_prefix_attn_workspace.argtypes = [KV, I64, I32, I32, I64, I64, I64, I32, ctypes.POINTER(SZ)]
            L.moe_prefix_attn.restype = ctypes.c_int
            L.moe_prefix_attn.argtypes = [KV, BA, P, I64, I64, I64, I64, HD, I32, HD, P, F32, ctypes.c_uint32, P, SZ, P]
            L.moe_status_string.restype = ctypes.c_char_p
            L.moe_status_string.argtypes = [ctypes.c_int]
            L.moe_version.restype = ctypes.c_char_p
            L.moe_version.argtypes = []
            _lib = L
    return _lib


def _check(fn: str, st: int):
    if st != MOE_OK:
        raise MoeError(fn, st)


def _ref(x):
    """A structure argument: a ctypes structure, or the bytes of one."""
    return x if type(x) is bytes else ctypes.byref(x)


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def status_string(status: int) -> str:
    try:
        return moe_status_string(status)
    except Exception:  # library not loadable: name only
        return STATUS_NAMES.get(status, str(status))


def moe_version() -> str:
    return lib().moe_version().decode()


def moe_plan_create(cfg: moe_config, weights: moe_weights):
    """Returns (plan handle, workspace bytes)."""
    plan = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check("moe_plan_create", lib().moe_plan_create(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(plan),
                                                    ctypes.byref(ws)))
    return plan, ws.value


def moe_plan_destroy(plan) -> None:
    lib().moe_plan_destroy(plan)


def moe_workspace_init(plan, ws_ptr: int, ws_bytes: int, stream: int) -> None:
    _check("moe_workspace_init", lib().moe_workspace_init(plan, ws_ptr, ws_bytes, stream))


def moe_workspace_check(plan, ws_ptr: int, ws_bytes: int, stream: int) -> int:
    """MOE_OK or MOE_ERR_WAIT (returned, not raised); raises on other statuses."""
    st = lib().moe_workspace_check(plan, ws_ptr, ws_bytes, stream)
    if st not in (MOE_OK, MOE_ERR_WAIT):
        raise MoeError("moe_workspace_check", st)
    return st


def moe_forward_prefill(plan, x_ptr: int, T: int, out_ptr: int, ws_ptr: int, ws_bytes: int, stream: int,
                        dbg: moe_debug_out | None = None) -> None:
    _check("moe_forward_prefill", lib().moe_forward_prefill(plan, x_ptr, T, out_ptr, ws_ptr, ws_bytes, stream,
                                                            ctypes.byref(dbg) if dbg is not None else None))


def moe_forward_decode(plan, x_ptr: int, out_ptr: int, ws_ptr: int, ws_bytes: int, stream: int,
                       dbg: moe_debug_out | None = None) -> None:
    _check("moe_forward_decode", lib().moe_forward_decode(plan, x_ptr, out_ptr, ws_ptr, ws_bytes, stream,
                                                          ctypes.byref(dbg) if dbg is not None else None))


def moe_forward_decode_batch(plan, x_ptr: int, T: int, out_ptr: int, ws_ptr: int, ws_bytes: int, stream: int,
                             dbg: moe_debug_out | None = None) -> None:
    _check("moe_forward_decode_batch", lib().moe_forward_decode_batch(plan, x_ptr, T, out_ptr, ws_ptr, ws_bytes,
                                                                      stream,
                                                                      ctypes.byref(dbg) if dbg is not None else None))


def moe_forward_decode_static(plan, x_ptr: int, out_ptr: int, stream: int, dbg: moe_debug_out | None = None) -> None:
    _check("moe_forward_decode_static", lib().moe_forward_decode_static(plan, x_ptr, out_ptr, stream,
                                                                        ctypes.byref(dbg) if dbg is not None else None))


def moe_gdn_scan(T: int, n_kheads: int, n_vheads: int, d_k: int, d_v: int, q_ptr: int, k_ptr: int, v_ptr: int,
                 alpha_ptr: int, beta_ptr: int, state_ptr: int, out_ptr: int, stream: int) -> None:
    _check("moe_gdn_scan", lib().moe_gdn_scan(T, n_kheads, n_vheads, d_k, d_v, q_ptr, k_ptr, v_ptr, alpha_ptr,
                                              beta_ptr, state_ptr, out_ptr, stream))


def moe_gdn_step(R: int, n_kheads: int, n_vheads: int, d_k: int, d_v: int, q_ptr: int, k_ptr: int, v_ptr: int,
                 alpha_ptr: int, beta_ptr: int, state_ptr: int, n_slots: int, slot_ptr: int, out_ptr: int,
                 stream: int) -> None:
    _check("moe_gdn_step", lib().moe_gdn_step(R, n_kheads, n_vheads, d_k, d_v, q_ptr, k_ptr, v_ptr, alpha_ptr,
                                              beta_ptr, state_ptr, n_slots, slot_ptr, out_ptr, stream))


def moe_rope_freqs(rot_dim: int, base: float, scaling: int = MOE_ROPE_NONE, factor: float = 1.0, trained: int = 1):
    """Returns (list of rot_dim / 2 frequencies, mscale)."""
    out = (ctypes.c_double * max(1, rot_dim // 2))()
    mscale = ctypes.c_float()
    _check("moe_rope_freqs", lib().moe_rope_freqs(rot_dim, base, scaling, factor, trained, out, ctypes.byref(mscale)))
    return list(out), mscale.value


def moe_rope_append(kv: moe_paged_kv, batch: moe_batch, T: int, q: moe_heads, q_out: moe_heads, n_heads: int,
                    k: moe_heads, v: moe_heads, pos_ptr: int | None, inv_freq_ptr: int | None, rot_dim: int,
                    mscale: float, flags: int, stream: int) -> None:
    st = (_lib or lib()).moe_rope_append(_ref(kv), _ref(batch), T, _ref(q), _ref(q_out), n_heads, _ref(k), _ref(v),
                                         pos_ptr, inv_freq_ptr, rot_dim, mscale, flags, stream)
    if st:
        raise MoeError("moe_rope_append", st)


def moe_paged_attn_workspace(kv: moe_paged_kv, T: int, n_seqs: int, max_q: int, max_kv: int, n_heads: int,
                             window: int = 0) -> int:
    n = ctypes.c_size_t()
    st = (_lib or lib()).moe_paged_attn_workspace(_ref(kv), T, n_seqs, max_q, max_kv, n_heads, window, ctypes.byref(n))
    if st:
        raise MoeError("moe_paged_attn_workspace", st)
    return n.value


def moe_paged_attn(kv: moe_paged_kv, batch: moe_batch, T: int, max_q: int, max_kv: int, q: moe_heads, n_heads: int,
                   out: moe_heads, lse_ptr: int | None, scale: float, window: int, flags: int, ws_ptr: int | None,
                   ws_bytes: int, stream: int) -> None:
    st = (_lib or lib()).moe_paged_attn(_ref(kv), _ref(batch), T, max_q, max_kv, _ref(q), n_heads, _ref(out), lse_ptr,
                                        scale, window, flags, ws_ptr, ws_bytes, stream)
    if st:
        raise MoeError("moe_paged_attn", st)


def moe_prefix_attn_workspace(kv: moe_paged_kv, T: int, n_seqs: int, n_groups: int, max_q: int, max_prefix: int,
                              max_suffix: int, n_heads: int) -> int:
    n = ctypes.c_size_t()
    st = (_lib or lib()).moe_prefix_attn_workspace(_ref(kv), T, n_seqs, n_groups, max_q, max_prefix, max_suffix, n_heads,
                                                   ctypes.byref(n))
    if st:
        raise MoeError("moe_prefix_attn_workspace", st)
    return n.value


def moe_prefix_attn(kv: moe_paged_kv, batch: moe_batch, groups: moe_prefix_groups, T: int, max_q: int, max_prefix: int,
                    max_suffix: int, q: moe_heads, n_heads: int, out: moe_heads, lse_ptr: int | None, scale: float,
                    flags: int, ws_ptr: int | None, ws_bytes: int, stream: int) -> None:
    _check("moe_prefix_attn", (_lib or lib()).moe_prefix_attn(_ref(kv), _ref(batch), _opt(groups), T, max_q, max_prefix,
                                                              max_suffix, _ref(q), n_heads, _ref(out), lse_ptr, scale, flags,
                                                              ws_ptr, ws_bytes, stream))


def moe_pages_workspace(pages: moe_pages, n: int) -> int:
    size = ctypes.c_size_t()
    _check("moe_pages_workspace", lib().moe_pages_workspace(_ref(pages), n, size))
    return size.value


def moe_pages_grow(src: moe_pages, dst: moe_pages, n: int, seqs_ptr: int | None, tokens_ptr: int | None,
                   error_ptr: int, ws_ptr: int, ws_bytes: int, stream: int) -> None:
    st = (_lib or lib()).moe_pages_grow(_ref(src), _ref(dst), n, seqs_ptr, tokens_ptr, error_ptr, ws_ptr, ws_bytes, stream)
    if st:
        raise MoeError("moe_pages_grow", st)


def moe_pages_fork(src: moe_pages, dst: moe_pages, mem: moe_page_memory, n: int, src_ptr: int | None,
                   dst_ptr: int | None, error_ptr: int, ws_ptr: int, ws_bytes: int, stream: int) -> None:
    st = (_lib or lib()).moe_pages_fork(_ref(src), _ref(dst), _ref(mem), n, src_ptr, dst_ptr, error_ptr, ws_ptr, ws_bytes,
                                        stream)
    if st:
        raise MoeError("moe_pages_fork", st)


def moe_pages_free(src: moe_pages, dst: moe_pages, n: int, seqs_ptr: int | None, error_ptr: int, ws_ptr: int,
                   ws_bytes: int, stream: int) -> None:
    _check("moe_pages_free", lib().moe_pages_free(_ref(src), _ref(dst), n, seqs_ptr, error_ptr, ws_ptr, ws_bytes, stream))


def moe_pages_compact(src: moe_pages, dst: moe_pages, mem: moe_page_memory, error_ptr: int, ws_ptr: int,
                      ws_bytes: int, stream: int) -> None:
    _check("moe_pages_compact", lib().moe_pages_compact(_ref(src), _ref(dst), _ref(mem), error_ptr, ws_ptr, ws_bytes, stream))


def moe_pages_copy(mem: moe_page_memory, n_pages: int, n: int, src_ptr: int | None, dst_ptr: int | None,
                   stream: int) -> None:
    _check("moe_pages_copy", lib().moe_pages_copy(_ref(mem), n_pages, n, src_ptr, dst_ptr, stream))


def moe_pages_check(error_ptr: int, stream: int) -> int:
    """The first error that the pool's calls left (MOE_OK, MOE_ERR_SHAPE or MOE_ERR_ALLOC: returned,
    not raised); raises on other statuses."""
    st = lib().moe_pages_check(error_ptr, stream)
    if st not in (MOE_OK, MOE_ERR_SHAPE, MOE_ERR_ALLOC):
        raise MoeError("moe_pages_check", st)
    return st


def _opt(x):
    return None if x is None else _ref(x)


def moe_rms_norm(T: int, n_heads: int, width: int, dtype: int, x: moe_heads, residual: moe_heads | None,
                 sum: moe_heads | None, weight_ptr: int | None, offset: float, eps: float, out_dtype: int, out: moe_heads,
                 group: int, scale_ptr: int | None, stream: int) -> None:
    _check("moe_rms_norm", lib().moe_rms_norm(T, n_heads, width, dtype, _opt(x), _opt(residual), _opt(sum), weight_ptr, offset,
                                              eps, out_dtype, _opt(out), group, scale_ptr, stream))


def moe_linear(w: moe_linear_weights, T: int, x_ptr: int | None, x_stride: int, x_dtype: int, x_scale_ptr: int | None,
               x_group: int, out_ptr: int | None, out_stride: int, out_dtype: int, stream: int) -> None:
    _check("moe_linear", lib().moe_linear(_opt(w), T, x_ptr, x_stride, x_dtype, x_scale_ptr, x_group, out_ptr, out_stride,
                                          out_dtype, stream))


def moe_sample_workspace(R: int, V: int) -> int:
    size = ctypes.c_size_t()
    _check("moe_sample_workspace", (_lib or lib()).moe_sample_workspace(R, V, size))
    return size.value


def moe_sample(R: int, V: int, logits_ptr: int | None, row_stride: int, dtype: int, u_ptr: int | None,
               temperature_ptr: int | None, top_k_ptr: int | None, top_p_ptr: int | None, min_p_ptr: int | None,
               token_ptr: int | None, prob_ptr: int | None, ws_ptr: int | None, ws_bytes: int, stream: int) -> None:
    _check("moe_sample", lib().moe_sample(R, V, logits_ptr, row_stride, dtype, u_ptr, temperature_ptr, top_k_ptr, top_p_ptr,
                                          min_p_ptr, token_ptr, prob_ptr, ws_ptr, ws_bytes, stream))


def moe_pack_qparams(src_ptr: int, dst_ptr: int, rows: int, k: int, stream: int) -> None:
    _check("moe_pack_qparams", lib().moe_pack_qparams(src_ptr, dst_ptr, rows, k, stream))


def moe_pack_codes(src_ptr: int, dst_ptr: int, rows: int, k: int, stream: int) -> None:
    _check("moe_pack_codes", lib().moe_pack_codes(src_ptr, dst_ptr, rows, k, stream))


# ---------------------------------------------------------------- HIP events (timing)

_hip = None


def hip() -> ctypes.CDLL:
    global _hip
    if _hip is None:
        h = ctypes.CDLL("libamdhip64.so")
        P = ctypes.c_void_p
        h.hipEventCreate.argtypes = [ctypes.POINTER(P)]
        h.hipEventRecord.argtypes = [P, P]
        h.hipEventSynchronize.argtypes = [P]
        h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), P, P]
        h.hipEventDestroy.argtypes = [P]
        _hip = h
    return _hip


class HipEvents:
    """An array of hipEvent_t usable as moe_debug_out.events."""

    def __init__(self, n: int):
        self.n = n
        self.arr = (ctypes.c_void_p * n)()
        for i in range(n):
            ev = ctypes.c_void_p()
            if hip().hipEventCreate(ctypes.byref(ev)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.arr[i] = ev.value

    @property
    def ptr(self) -> int:
        return ctypes.addressof(self.arr)

    def record(self, i: int, stream: int) -> None:
        if hip().hipEventRecord(self.arr[i], stream) != 0:
            raise RuntimeError("hipEventRecord failed")

    def elapsed_ms(self, i: int, j: int) -> float:
        ms = ctypes.c_float()
        hip().hipEventSynchronize(self.arr[j])
        if hip().hipEventElapsedTime(ctypes.byref(ms), self.arr[i], self.arr[j]) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return ms.value

    def close(self) -> None:
        for i in range(self.n):
            if self.arr[i]:
                hip().hipEventDestroy(self.arr[i])
                self.arr[i] = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
