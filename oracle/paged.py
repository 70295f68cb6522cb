"""fp64 restatement of the paged key/value cache: append, attention, eviction.

Plain numpy, one sequence and one row at a time; bf16 values come in as
float64 and results stay float64 (the caller rounds).  Test infrastructure.
"""

from __future__ import annotations

import numpy as np

__all__ = ["slot_rows", "cache_append", "paged_attention", "cache_evict"]


def slot_rows(table_row, n, page):
    """(page number, row inside the page) of slots 0..n-1 of one sequence."""
    t = np.arange(n)
    return np.asarray(table_row)[t // page], t % page


def cache_append(k_new, v_new, k_pages, v_pages, table, lens, cu, pos=None, theta=500000.0):
    """Copies of the pages with the new rows in place; rows without a slot are dropped."""
    K, V = k_pages.copy(), v_pages.copy()
    page, d = K.shape[1], K.shape[3]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t = lens[b] - n + i
            if t < 0:
                continue
            k = k_new[cu[b] + i].copy()
            if pos is not None:
                ang = float(pos[cu[b] + i]) * float(theta) ** (-2.0 * np.arange(d // 2) / d)
                lo, hi = k[:, :d // 2].copy(), k[:, d // 2:].copy()
                k[:, :d // 2] = lo * np.cos(ang) - hi * np.sin(ang)
                k[:, d // 2:] = hi * np.cos(ang) + lo * np.sin(ang)
            p, r = table[b][t // page], t % page
            K[p, r], V[p, r] = k, v_new[cu[b] + i]
    return K, V


def paged_attention(q, k_pages, v_pages, table, lens, cu, scale=None, heads_scored=None):
    """For every packed row and head: o, lse, and the sizes that bound rounding.

    Returns a dict of o [T, Hq, d]; lse [T, Hq]; av = sum_t p_t |v_t| [T, Hq, d];
    aqk = scale * max over visible t of sum_e |q_e k_te| [T, Hq]; with heads_scored (1 or
    Hkv) also weights [B, heads_scored, max len]: what this call adds to them.
    """
    T, Hq, d = q.shape
    page, Hkv = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    o, av = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse, aqk = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    w = np.zeros((len(lens), heads_scored or 1, max(max(lens), 1)))
    for b in range(len(lens)):
        p, r = slot_rows(table[b], lens[b], page)
        K, V = k_pages[p, r], v_pages[p, r]
        n = cu[b + 1] - cu[b]
        for i in range(n):
            end = lens[b] - n + i + 1
            if end <= 0:
                continue
            for h in range(Hq):
                k, v, x = K[:end, h // G], V[:end, h // G], q[cu[b] + i, h]
                s = (k @ x) * scale
                top = s.max()
                e = np.exp(s - top)
                a = e / e.sum()
                row = cu[b] + i
                o[row, h], av[row, h] = a @ v, a @ np.abs(v)
                lse[row, h] = top + np.log(e.sum())
                aqk[row, h] = (np.abs(k) @ np.abs(x)).max() * scale
                w[b, h // G if w.shape[1] > 1 else 0, :end] += a
    return dict(o=o, lse=lse, av=av, aqk=aqk, weights=w)


def cache_evict(k_pages, v_pages, table, lens, weights, keep, sink, recent, dst_table, out_width):
    """(K, V, weights_out, new_lens, kept): copies of the pages with the kept rows in dst_table's pages."""
    K, V = k_pages.copy(), v_pages.copy()
    page, Hkv = K.shape[1], K.shape[2]
    B, Hs = weights.shape[:2]
    w_out = np.zeros((B, Hs, out_width))
    kept = np.full((B, Hs, keep), -1, dtype=np.int64)
    new = [min(int(n), keep) for n in lens]
    for b in range(B):
        n = int(lens[b])
        p, r = slot_rows(table[b], n, page)
        dp, dr = slot_rows(dst_table[b], new[b], page)
        for h in range(Hs):
            safe = lambda j: j < sink or j >= n - recent  # noqa: E731
            order = sorted(range(n), key=lambda j: (not safe(j), -(weights[b, h, j] + 0.0), j))
            idx = np.array(sorted(order[:keep]), dtype=np.int64)
            kept[b, h, :len(idx)] = idx
            w_out[b, h, :len(idx)] = weights[b, h, idx]
            g = slice(h, h + 1) if Hs > 1 or Hkv == 1 else slice(None)
            K[dp, dr, g], V[dp, dr, g] = k_pages[p[idx], r[idx], g], v_pages[p[idx], r[idx], g]
    return K, V, w_out, new, kept
