"""Forking, giving back, compacting and copying the pages of the paged
key/value cache, entry by entry from the definitions.  Arguments are not
modified.  ``fits`` says whether everything fitted."""
from __future__ import annotations

import numpy as np


def fork(page, table, shares, free, count, src, dst, length):
    """(table, shares, free_left, copies, fits); copies: (from, to) pairs."""
    table, shares = np.array(table, dtype=np.int64), np.array(shares, dtype=np.int64)
    rows, width = table.shape
    left, copies = min(max(int(count), 0), len(free)), []
    whole = list(zip(map(int, src), map(int, dst), map(int, length)))
    bad = left != count or len({d for _, d, _ in whole}) < len(whole) or bool({d for _, d, _ in whole} & {s for s, _, _ in whole})
    for s, d, n in whole:
        bad |= not (0 <= s < rows and 0 <= d < rows and 0 <= n <= width * page)
        if not bad and n % page:
            bad |= not 0 <= table[s, n // page] < len(shares)
    fresh = sum(n % page > 0 for _, _, n in whole)
    bad |= fresh > left or not all(0 <= int(p) < len(shares) for p in free[max(left - fresh, 0):left])
    if bad:
        return table, shares, left, [], False
    fits = True
    for s, d, n in whole:
        for col in range(-(-n // page)):
            e = int(table[s, col])
            if n // page == col:
                left -= 1
                copies.append((e, int(free[left])))
                e = int(free[left])
            elif e >= len(shares):
                fits, e = False, -1
            elif e >= 0:
                shares[e] += 1
            table[d, col] = e
    return table, shares, left, copies, fits


def give_back(table, shares, free, count, first, end):
    """(table, shares, free, free_left, fits)."""
    table, shares, free = (np.array(x, dtype=np.int64) for x in (table, shares, free))
    rows, width = table.shape
    at, fits, owners = min(max(int(count), 0), len(free)), True, shares + 1
    fits = at == count
    gone = set()
    for r in range(rows):
        a, b = int(first[r]), int(end[r])
        if b <= a:
            continue
        if a < 0 or b > width:
            fits = False
            continue
        for col in range(a, b):
            e = int(table[r, col])
            if e < 0:
                continue
            table[r, col] = -1
            if e >= len(shares):
                fits = False
                continue
            owners[e] -= 1
            fits &= owners[e] >= 0
            if owners[e] <= 0:
                gone.add(e)
    for p in sorted(gone, reverse=True):
        owners[p] = 1
        if at < len(free):
            free[at] = p
            at += 1
        else:
            fits = False
    return table, owners - 1, free, at, fits


def compact(page, table, shares, free, count, kv_len):
    """(table, shares, free, page_map, copies, fits)."""
    table, shares, free = (np.array(x, dtype=np.int64) for x in (table, shares, free))
    pages, count = len(shares), int(count)
    listed = [int(p) for p in free[:max(count, 0)]]
    if not 0 <= count <= pages or len(set(listed)) < len(listed) or not all(0 <= p < pages for p in listed):
        for p in listed if 0 <= count <= pages else []:
            if 0 <= p < pages:
                shares[p] = 0
        return table, shares, free, np.arange(pages), [], False
    used, gone = pages - count, set(listed)
    copies = list(zip((p for p in range(used, pages) if p not in gone), (p for p in range(used) if p in gone)))
    page_map = np.array([-1 if p in gone else p for p in range(pages)])
    for p in gone:
        shares[p] = 0
    for a, b in copies:
        page_map[a], shares[b], shares[a] = b, shares[a], 0
    moved, fits = dict(copies), True
    for r in range(table.shape[0]):
        n = int(kv_len[r])
        if not 0 <= n <= table.shape[1] * page:
            fits = False
            continue
        for col in range(-(-n // page)):
            e = int(table[r, col])
            fits &= e < pages and e not in gone
            table[r, col] = moved.get(e, e)
    free[:count] = np.arange(pages - 1, used - 1, -1)
    return table, shares, free, page_map, copies, fits
