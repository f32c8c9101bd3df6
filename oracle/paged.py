"""Plain NumPy forms of the paged-cache operators: whole numbers exactly, attention in fp64.
Test infrastructure only."""
from __future__ import annotations

import numpy as np

INV127 = np.float32(1.0) / np.float32(127.0)


def page_plan(old, new, table, ring, state, P, max_tokens):
    """The plan, sequence by sequence. Returns (len_out, slots, cu, state, status, table, ring)."""
    table, ring = table.copy(), ring.copy()
    B, cols = table.shape
    n = len(ring)
    head, count = int(state[0]) % n, min(max(int(state[1]), 0), n)
    len_out, slots = np.array(old, np.int32), np.full(max_tokens, -1, np.int32)
    cu = np.zeros(B + 1, np.int32)
    taken = total = freed = denied = 0
    full = False
    back = []
    for b in range(B):
        o, w = min(max(int(old[b]), 0), cols * P), int(new[b])
        len_out[b] = o
        cu[b] = total
        if w < 0 or w > cols * P:
            denied += 1
            continue
        n0, n1 = -(-o // P), -(-w // P)
        if w > o:
            if full or taken + n1 - n0 > count or total + w - o > max_tokens:
                full = True
                denied += 1
                continue
            for lp in range(n0, n1):
                table[b, lp] = ring[(head + taken) % n]
                taken += 1
            for pos in range(o, w):
                page = table[b, pos // P]
                slots[total] = page * P + pos % P if 0 <= page < n else -1
                total += 1
        else:
            back += [table[b, lp] for lp in range(n1, n0)]
        len_out[b] = w
    cu[B] = total
    for page in back:
        ring[(head + count + freed) % n] = page
        freed += 1
    return (len_out, slots, cu, np.array([(head + taken) % n, count - taken + freed], np.int32),
            np.array([total, taken, freed, denied], np.int32), table, ring)


def page_summary(rows):
    """Codes and scale of one page's rows [P][d] (fp32 values)."""
    mean = (rows.astype(np.float64).sum(0) / len(rows)).astype(np.float32)
    if not np.isfinite(mean).all():
        return np.zeros(len(mean), np.int8), np.float32(np.nan)
    scale = np.float32(np.abs(mean).max()) * INV127
    if scale == 0:
        return np.zeros(len(mean), np.int8), scale
    return np.clip(np.rint(mean / scale), -127, 127).astype(np.int8), scale


def page_scores(q, codes, scales):
    """Scores of pages for one KV head: q fp32 [G][d], codes [n][d], scales [n]."""
    best = np.full(len(codes), -np.inf, np.float32)
    for row in q:
        s = np.float32(np.abs(row).max()) * INV127
        ok = np.isfinite(row).all() and s > 0
        c = np.clip(np.rint(row / s), -127, 127).astype(np.int64) if ok else np.zeros(len(row), np.int64)
        dot = (codes.astype(np.int64) @ c).astype(np.float32)
        with np.errstate(invalid="ignore"):
            best = np.fmax(best, dot * (s if np.isfinite(row).all() else np.float32(0)) * scales)
    best[np.isnan(scales)] = np.inf
    return best


def page_select(q, codes, scales, table, L, P, n_pages, k, first, last):
    """Selected pages [n_kv][k] of one sequence."""
    n_kv = codes.shape[1]
    G = len(q) // n_kv
    n = -(-L // P)
    sel = np.full((n_kv, k), -1, np.int32)
    for g in range(n_kv):
        if n <= k:
            sel[g, :n] = np.arange(n)
            continue
        pages = table[:n]
        ok = (pages >= 0) & (pages < n_pages)
        at = np.where(ok, pages, 0)
        s = np.where(ok, page_scores(q[g * G:(g + 1) * G], codes[at, g], scales[at, g]), -np.inf)
        i = np.arange(n)
        kept = (i < first) | (i >= n - last)
        # kept pages first, then by score, then by page
        sel[g] = np.sort(np.lexsort((i, -(s + 0.0), ~kept))[:k])
    return sel


def paged_attention(q, k, v, table, L, scale, window=0, pages=None):
    """One sequence: q [H][d], k / v [n_pages][P][n_kv][d] fp64. Returns (out, lse)."""
    n_pages, P, n_kv, d = k.shape
    H = len(q)
    G = H // n_kv
    out, lse = np.zeros((H, d)), np.full(H, -np.inf)
    L = min(max(int(L), 0), len(table) * P)
    lo = max(0, L - window) if window else 0
    for g in range(n_kv):
        listed = range(-(-L // P)) if pages is None else [p for p in pages[g] if 0 <= p < len(table)]
        rows, vals = [], []
        for lp in listed:
            page = table[lp]
            if not 0 <= page < n_pages:
                continue
            a, e = max(lo - lp * P, 0), min(L - lp * P, P)
            if e > a:
                rows.append(k[page, a:e, g])
                vals.append(v[page, a:e, g])
        if not rows:
            continue
        kk, vv = np.concatenate(rows), np.concatenate(vals)
        s = scale * (q[g * G:(g + 1) * G].astype(np.float64) @ kk.T)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        out[g * G:(g + 1) * G] = p @ vv / p.sum(1, keepdims=True)
        lse[g * G:(g + 1) * G] = (m + np.log(p.sum(1, keepdims=True)))[:, 0]
    return out, lse
