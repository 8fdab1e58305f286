"""Paged key/value cache: block tables and slot maps from request lengths, the
cache write, and attention of new tokens over the cache, in float64 (integers
for the plan), token by token from the definitions."""
from __future__ import annotations

import numpy as np


def plan(page, cached, fresh, free_pages, free_count, table, tokens):
    """One step's plan.  ``table`` (requests, width) is not modified.  Returns
    (q_start, kv_len, table, slots, positions, free_left, fits); tokens
    without a page have slot -1, as have the slots up to ``tokens``."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    left, fits = int(free_count), True
    slots = np.full(tokens, -1, dtype=np.int64)
    positions = np.zeros(tokens, dtype=np.int64)
    q_start, kv_len, t = [0], [], 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        c, f = int(c), int(f)
        if c < 0 or f < 0 or c + f > width * page or c + f > 2 ** 31 - 1:
            fits, f, c = False, 0, min(max(c, 0), width * page)
        for p in range(c, c + f):
            col = p // page
            if p == c and c % page:
                pass  # falls into the partly filled page
            elif p % page == 0:
                if left > 0:
                    left -= 1
                    table[b, col] = free_pages[left]
                else:
                    fits, table[b, col] = False, -1
            if t < tokens:
                positions[t] = p
                if table[b, col] >= 0:
                    slots[t] = table[b, col] * page + p % page
            else:
                fits = False
            t += 1
        q_start.append(t)
        kv_len.append(c + f)
    return np.array(q_start), np.array(kv_len, dtype=np.int64), table, slots, positions, left, fits


def store(pool, new, slots):
    """pool (page, token, head, column) with row t of ``new`` written to slot slots[t] (< 0: skipped)."""
    out = np.array(pool)
    page = out.shape[1]
    for t, s in enumerate(slots):
        if s >= 0:
            out[s // page, s % page] = new[t]
    return out


def attention(q, k_pool, v_pool, table, q_start, kv_len, scale):
    """q (token, head, column), pools (page, token, kv head, column).  Returns
    (o, lse, absum, amax): absum = sum_k p_k |v_k| and amax = max_k scale
    sum_c |q_c k_kc| of each row's keys, for error bounds.  Rows of no request
    and rows without keys: o = 0, lse = -inf."""
    tokens, heads, d = q.shape
    page, kv_heads = k_pool.shape[1], k_pool.shape[2]
    g = heads // kv_heads
    o = np.zeros((tokens, heads, d))
    absum = np.zeros((tokens, heads, d))
    lse = np.full((tokens, heads), -np.inf)
    amax = np.zeros((tokens, heads))
    for b in range(len(kv_len)):
        q0, q1, kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if q1 == q0 or kv <= 0:
            continue
        pages = [int(x) for x in table[b][:-(-kv // page)]]
        k = np.concatenate([k_pool[p] for p in pages])[:kv].astype(np.float64)
        v = np.concatenate([v_pool[p] for p in pages])[:kv].astype(np.float64)
        for j in range(q1 - q0):
            n = kv - (q1 - q0) + j + 1  # keys this row sees
            if n <= 0:
                continue
            for i in range(heads):
                kk, vv = k[:n, i // g], v[:n, i // g]
                x = q[q0 + j, i].astype(np.float64)
                s = scale * (kk @ x)
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                o[q0 + j, i] = p @ vv
                absum[q0 + j, i] = p @ np.abs(vv)
                lse[q0 + j, i] = m + np.log(e.sum())
                amax[q0 + j, i] = scale * (np.abs(kk) @ np.abs(x)).max()
    return o, lse, absum, amax
