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


class Pool:
    """The paged cache's bookkeeping by its definition in ``include/pages.h``.  cache: an array
    [plane][page] of page contents.  A call with an error changes nothing and returns its name."""

    def __init__(self, table, lens, refs, page_size, cache=None):
        self.table, self.lens, self.refs = (np.array(x, np.int64) for x in (table, lens, refs))
        self.page, self.cache = page_size, None if cache is None else np.array(cache)

    def _count(self, n):
        return -(-int(n) // self.page)

    def _fresh(self, n):
        return [p for p in range(len(self.refs)) if self.refs[p] <= 0][:n]

    def _known(self, seqs):
        cap = self.table.shape[1] * self.page
        return all(0 <= s < len(self.lens) and 0 <= self.lens[s] <= cap for s in seqs)

    def _held(self, s):
        return self.table[s, :self._count(self.lens[s])]

    def _sound(self, seqs):
        return all(((self._held(s) >= 0) & (self._held(s) < len(self.refs))).all() for s in seqs)

    def grow(self, seqs, tokens):
        if len(set(seqs)) != len(seqs) or not self._known(seqs):
            return "shape"
        cap = self.table.shape[1] * self.page
        if any(t < 0 or self.lens[s] + t > cap for s, t in zip(seqs, tokens)):
            return "shape"
        need = [self._count(self.lens[s] + t) - self._count(self.lens[s]) for s, t in zip(seqs, tokens)]
        fresh = self._fresh(sum(need))
        if len(fresh) < sum(need):
            return "alloc"
        for s, t, n in zip(seqs, tokens, need):
            at = self._count(self.lens[s])
            for c in range(n):
                p = fresh.pop(0)
                self.table[s, at + c], self.refs[p] = p, 1
            self.lens[s] += t
        return ""

    def fork(self, src, dst):
        if not self._known(src) or not self._known(dst) or len(set(dst)) != len(dst) or set(src) & set(dst):
            return "shape"
        if any(self.lens[d] != 0 for d in dst) or not self._sound(src):
            return "shape"
        part = [s for s in src if self.lens[s] % self.page]
        fresh = self._fresh(len(part))
        if len(fresh) < len(part):
            return "alloc"
        for s, d in zip(src, dst):
            full = int(self.lens[s]) // self.page
            for c in range(full):
                self.table[d, c] = self.table[s, c]
                self.refs[self.table[s, c]] += 1
            if self.lens[s] % self.page:
                p = fresh.pop(0)
                self.cache[:, p] = self.cache[:, self.table[s, full]]
                self.table[d, full], self.refs[p] = p, 1
            self.lens[d] = self.lens[s]
        return ""

    def free(self, seqs):
        if len(set(seqs)) != len(seqs) or not self._known(seqs) or not self._sound(seqs):
            return "shape"
        for s in seqs:
            for p in self._held(s):
                self.refs[p] -= 1
            self.lens[s] = 0
        return ""

    def compact(self):
        every = range(len(self.lens))
        if not self._known(every) or not self._sound(every):
            return "shape"
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        move = [p for p in used if p >= len(used)]
        hole = [p for p in range(len(used)) if self.refs[p] <= 0]
        to = dict(zip(move, hole))
        for a, b in to.items():
            self.cache[:, b] = self.cache[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in every:
            for c in range(self._count(self.lens[s])):
                self.table[s, c] = to.get(int(self.table[s, c]), self.table[s, c])
        return ""
