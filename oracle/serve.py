"""Plain binary64 forms of the serving operators (numpy): rotary append, paged attention, gated
delta steps.  Written from the definitions in ``include/attn.h`` and ``include/gdn.h``; shares no
code with the library.  16-bit values are passed as float arrays."""

from __future__ import annotations

import numpy as np


def rope(x, pos, inv_freq, mscale=1.0, interleaved=False):
    """x: [T][heads][D]; pos: [T]; the first 2 len(inv_freq) elements of each head rotated."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = len(inv_freq)
    th = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(th[:, i])[:, None], np.sin(th[:, i])[:, None]
        y[:, :, a] = mscale * (x[:, :, a] * c - x[:, :, b] * s)
        y[:, :, b] = mscale * (x[:, :, a] * s + x[:, :, b] * c)
    return y


def places(q_start, kv_len, table, page_size, n_pages, row=None):
    """Per token of the batch: (sequence, position, page or -1, offset)."""
    out = []
    for b in range(len(q_start) - 1):
        r = b if row is None else int(row[b])
        ok = 0 <= r < len(table)
        n = int(q_start[b + 1] - q_start[b])
        for i in range(n):
            p = (int(kv_len[r]) if ok else 0) - n + i
            page = -1
            if ok and p >= 0 and p // page_size < table.shape[1]:
                page = int(table[r, p // page_size])
                page = page if 0 <= page < n_pages else -1
            out.append((b, p, page, p % page_size))
    return out


def rope_append(q, k, v, k_cache, v_cache, table, q_start, kv_len, inv_freq, mscale=1.0, interleaved=False, pos=None,
                row=None):
    """Returns (q rotated, k_cache, v_cache) in binary64; the caches are [page][token][head][D]."""
    pl = places(q_start, kv_len, table, k_cache.shape[1], k_cache.shape[0], row)
    n = len(pl)
    pp = np.array([p for _, p, _, _ in pl]) if pos is None else np.asarray(pos)[:n]
    kc, vc = np.asarray(k_cache, np.float64).copy(), np.asarray(v_cache, np.float64).copy()
    qr = np.asarray(q, np.float64).copy()
    if n:
        qr[:n] = rope(q[:n], pp, inv_freq, mscale, interleaved)
        kr = rope(k[:n], pp, inv_freq, mscale, interleaved)
        for t, (_, _, page, off) in enumerate(pl):
            if page >= 0:
                kc[page, off], vc[page, off] = kr[t], v[t]
    return qr, kc, vc


def paged_attn(q, k_cache, v_cache, table, q_start, kv_len, scale, window=0, full=False, row=None):
    """Returns (out, lse, mass, spread): mass = sum_j softmax_j |v_j|, spread = the largest
    sum_i |q_i k_ji| of a visible key; rows behind the batch are NaN."""
    T, H, D = q.shape
    n_pages, ps, hk, _ = k_cache.shape
    out = np.full((T, H, D), np.nan)
    mass = np.full((T, H, D), np.nan)
    lse, spread = np.full((T, H), np.nan), np.zeros((T, H))
    for b in range(len(q_start) - 1):
        r = b if row is None else int(row[b])
        ok = 0 <= r < len(table)
        n, t0 = int(q_start[b + 1] - q_start[b]), int(q_start[b])
        total = int(kv_len[r]) if ok else 0
        length = max(0, min(total, table.shape[1] * ps))
        keys = []
        for j in range(length):
            page = int(table[r, j // ps])
            if 0 <= page < n_pages:
                keys.append((j, page, j % ps))
        kj = np.array([j for j, _, _ in keys], np.int64)
        idx = (np.array([p for _, p, _ in keys], np.int64), np.array([o for _, _, o in keys], np.int64))
        for i in range(n):
            p = total - n + i
            see = np.ones(len(kj), bool) if full else kj <= p
            if window:
                see &= kj > p - window
            for h in range(H):
                if not see.any():
                    out[t0 + i, h], mass[t0 + i, h], lse[t0 + i, h] = 0.0, 0.0, -np.inf
                    continue
                K = np.asarray(k_cache[idx[0][see], idx[1][see], h // (H // hk)], np.float64)
                V = np.asarray(v_cache[idx[0][see], idx[1][see], h // (H // hk)], np.float64)
                qq = np.asarray(q[t0 + i, h], np.float64)
                s = scale * (K @ qq)
                m = s.max()
                w = np.exp(s - m)
                out[t0 + i, h] = w @ V / w.sum()
                mass[t0 + i, h] = w @ np.abs(V) / w.sum()
                lse[t0 + i, h] = m + np.log(w.sum())
                spread[t0 + i, h] = (np.abs(K) @ np.abs(qq)).max()
    return out, lse, mass, spread


def gdn_step(q, k, v, alpha, beta, state, slot):
    """Returns (out, state) in binary64; rows in order."""
    S = np.asarray(state, np.float64).copy()
    R, hv, d = v.shape
    g = hv // k.shape[1]
    out = np.zeros((R, hv, d))
    for r in range(R):
        if not 0 <= int(slot[r]) < len(S):
            continue
        for h in range(hv):
            kk, qq = np.asarray(k[r, h // g], np.float64), np.asarray(q[r, h // g], np.float64)
            a, b = float(alpha[r, h]), float(beta[r, h])
            A = S[slot[r], h]
            A = a * (A - b * np.outer(A @ kk, kk)) + b * np.outer(np.asarray(v[r, h], np.float64), kk)
            S[slot[r], h] = A
            out[r, h] = A @ qq
    return out, S
