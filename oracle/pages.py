"""The cache's rows and pages by their definitions, one request, one token, one page after the
other, on integers.
"""
from __future__ import annotations

import numpy as np

__all__ = ["compact", "copy_pages", "resize", "select"]


def _holds(n, page_size):
    return -(-n // page_size)


def compact(cache, page_table, kv_len, cu_q, path, accepted, page_size):
    """cache [L, slots, ..] -> (the cache afterwards, new_len): token context + path[b, i] takes
    place context + i, as long as the path ascends inside the block."""
    after, new_len = cache.copy(), np.zeros(len(kv_len), np.int64)
    pages = cache.shape[1] // page_size
    width = page_table.shape[1]
    for b in range(len(kv_len)):
        n = int(cu_q[b + 1]) - int(cu_q[b])
        kv = min(max(int(kv_len[b]), 0), width * page_size)

        def slot(key):
            p = int(page_table[b, key // page_size]) if 0 <= key < kv else -1
            return p * page_size + key % page_size if 0 <= p < pages else -1

        taken, last = 0, -1
        for i in range(min(max(int(accepted[b]), 0), path.shape[1])):
            node = int(path[b, i])
            if not last < node < n:
                break
            src, dst = slot(kv - n + node), slot(kv - n + i)
            if src >= 0 and dst >= 0:
                after[:, dst] = cache[:, src]
            taken, last = i + 1, node
        new_len[b] = max(kv - n + taken, 0)
    return after, new_len


def copy_pages(cache, copies, page_size):
    after = cache.copy()
    pages = cache.shape[1] // page_size
    for src, dst in np.asarray(copies).tolist():
        if 0 <= src < pages and 0 <= dst < pages:
            after[:, dst * page_size:(dst + 1) * page_size] = cache[:, src * page_size:(src + 1) * page_size]
    return after


def resize(page_table, kv_len, new_len, refs, page_size):
    """-> (page_table, kv_len, refs, copies, served) afterwards."""
    table, refs = np.array(page_table), np.array(refs)
    B, width = table.shape
    P = len(refs)
    was = [min(max(int(n), 0), width * page_size) for n in kv_len]
    now = [min(max(int(n), 0), width * page_size) for n in new_len]
    for b in range(B):
        for c in range(_holds(now[b], page_size), _holds(was[b], page_size)):
            if 0 <= table[b, c] < P:
                refs[table[b, c]] -= 1
            table[b, c] = -1
    free = [p for p in range(P) if refs[p] == 0]
    copies, served, out_of = np.full((B, 2), -1), np.ones(B, np.int64), False
    lens = list(was)
    for b in range(B):
        if now[b] > was[b]:
            hold, want = _holds(was[b], page_size), _holds(now[b], page_size)
            last = int(table[b, hold - 1]) if was[b] % page_size else -1
            shares = 0 <= last < P
            # the count as it was before this call's copies decides whether the request waits in line
            lined = shares and refs[last] + int((copies[:b, 0] == last).sum()) > 1
            copied = shares and refs[last] > 1
            need = want - hold + copied
            if (need or lined) and (out_of or need > len(free)):
                out_of, served[b] = True, 0
                continue
            if copied:
                refs[last] -= 1
                copies[b] = last, free.pop(0)
                table[b, hold - 1] = copies[b, 1]
                refs[copies[b, 1]] = 1
            for c in range(hold, want):
                table[b, c] = free.pop(0)
                refs[table[b, c]] = 1
        lens[b] = now[b]
    return table, np.array(lens), refs, copies, served


def select(page_table, kv_len, src, refs, page_size):
    """-> (new_table, new_len, refs)."""
    B, width = page_table.shape
    refs = np.array(refs)
    table, lens = np.full((len(src), width), -1), np.zeros(len(src), np.int64)

    def count(row, n, by):
        for p in row[:_holds(n, page_size)]:
            if 0 <= p < len(refs):
                refs[p] += by

    for r, b in enumerate(np.asarray(src).tolist()):
        if 0 <= b < B:
            lens[r] = min(max(int(kv_len[b]), 0), width * page_size)
            hold = _holds(int(lens[r]), page_size)
            table[r, :hold] = page_table[b, :hold]
            count(page_table[b], int(lens[r]), 1)
    for b in range(B):
        count(page_table[b], min(max(int(kv_len[b]), 0), width * page_size), -1)
    return table, lens, refs
