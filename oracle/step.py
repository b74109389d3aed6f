"""Plain binary64 forms of the operators around the mixers (numpy): norm with the residual's
addition, 4-bit projections, sampling.  Written from the definitions in ``include/norm.h``,
``include/linear.h`` and ``include/sample.h``; shares no code with the library.  16-bit values are
passed as float arrays."""

from __future__ import annotations

import numpy as np


def rms_norm(x, weight=None, eps=1e-6, offset=0.0, residual=None):
    """Returns (y, h)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    w = offset + (0.0 if weight is None else np.asarray(weight, np.float64))
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w, h


def group_scales(y, most, group=0):
    """Scales of the groups of y's rows (group 0: whole rows) whose codes reach up to `most`."""
    g = group or y.shape[-1]
    return np.abs(y.reshape(*y.shape[:-1], -1, g)).max(-1) / most


def unpack(codes):
    """4-bit codes of words [N][K / 8], element k in bits 4 (k % 8) of word k / 8."""
    c = np.asarray(codes).astype(np.int64) & 0xFFFFFFFF
    return np.stack([(c >> (4 * j)) & 15 for j in range(8)], -1).reshape(c.shape[0], -1)


def linear(x, codes, scale, bias, x_scale=None):
    """x W^T with W = scale * code + bias by groups of 64; returns (out, mass), mass = sum |x| |w|."""
    q = unpack(codes).astype(np.float64)
    w = q * np.repeat(np.asarray(scale, np.float64), 64, 1) + np.repeat(np.asarray(bias, np.float64), 64, 1)
    x = np.asarray(x, np.float64)
    if x_scale is not None:
        x = x * np.repeat(np.asarray(x_scale, np.float64), x.shape[1] // x_scale.shape[1], 1)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Returns (token, probability, slack): slack is the smallest distance, as a share of the mass that it is
    compared with, between a cumulative mass and the border that decides about it."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    top = l.max() if l.size else -np.inf
    if top == -np.inf:
        return -1, 0.0, 1.0
    first = int(np.argmax(l))
    if not temperature > 0:
        return first, 1.0, 1.0
    l = np.minimum(l, float(np.finfo(np.float32).max))
    far = np.where(l > -np.inf, l - l[first], 0.0) / (temperature if temperature < np.inf else 1e300)
    w = np.where(l > -np.inf, np.exp(far), 0.0)
    order = np.lexsort((np.arange(len(l)), -l))
    order = order[l[order] > -np.inf]
    slack = 1.0
    min_p = min(min_p, 1.0)
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        upto = np.cumsum(w[order])
        slack = min(slack, np.abs(upto / upto[-1] - top_p).min())
        order = order[:max(1, int((upto < top_p * upto[-1]).sum()) + 1)]
    if min_p > 0:
        near = np.abs(w[order] / min_p - 1)
        slack = min(slack, near[near > 0].min() if (near > 0).any() else 1.0)
    kept = np.sort(order[w[order] >= min_p] if min_p > 0 else order)
    upto = np.cumsum(w[kept])
    u = min(max(u, 0.0), 1.0) if u == u else 0.0
    slack = min(slack, np.abs(upto / upto[-1] - u).min())
    i = min(int((upto <= u * upto[-1]).sum()), int(np.flatnonzero(w[kept])[-1]))
    return int(kept[i]), float(w[kept[i]] / upto[-1]), float(slack)


def prefix_attn(q, k_cache, v_cache, table, q_start, kv_len, group_start, prefix_len, scale, full=False, row=None):
    """Returns (out, lse, mass, spread) as ``serve.paged_attn`` does."""
    T, H, D = q.shape
    n_pages, ps, hk, _ = k_cache.shape
    out, mass = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan)
    lse, spread = np.full((T, H), np.nan), np.zeros((T, H))

    def stored(r, a, b):
        """(position, page, offset) of the positions a .. b - 1 of table row r that have a place."""
        if not 0 <= r < len(table):
            return []
        b = min(b, table.shape[1] * ps)
        return [(j, int(table[r, j // ps]), j % ps) for j in range(a, b) if 0 <= table[r, j // ps] < n_pages]

    rows = list(range(len(q_start) - 1)) if row is None else [int(x) for x in row]
    for g in range(len(prefix_len)):
        prefix = max(int(prefix_len[g]), 0)
        for b in range(int(group_start[g]), int(group_start[g + 1])):
            r = rows[b]
            n, t0 = int(q_start[b + 1] - q_start[b]), int(q_start[b])
            total = int(kv_len[r]) if 0 <= r < len(table) else 0
            shared = stored(rows[int(group_start[g])], 0, prefix)
            own = stored(r, min(prefix, table.shape[1] * ps), max(total, 0))
            for i in range(n):
                keys = shared + [x for x in own if full or x[0] <= total - n + i]
                if not keys:
                    out[t0 + i], mass[t0 + i], lse[t0 + i] = 0.0, 0.0, -np.inf
                    continue
                at = tuple(np.array([x[c] for x in keys]) for c in (1, 2))
                for h in range(H):
                    K, V = (np.asarray(c[at[0], at[1], h // (H // hk)], np.float64) for c in (k_cache, v_cache))
                    s = scale * (K @ np.asarray(q[t0 + i, h], np.float64))
                    w = np.exp(s - s.max())
                    out[t0 + i, h], mass[t0 + i, h] = w @ V / w.sum(), w @ np.abs(V) / w.sum()
                    lse[t0 + i, h] = s.max() + np.log(w.sum())
                    spread[t0 + i, h] = (np.abs(K) @ np.abs(np.asarray(q[t0 + i, h], np.float64))).max()
    return out, lse, mass, spread
