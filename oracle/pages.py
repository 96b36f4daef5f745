"""The life of a paged cache's pages in plain Python: sequences forked, reordered and ended, the pages in use moved to
the front of the pool.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np


def held(length, P):
    return -(-max(int(length), 0) // P)


def fork(table, lengths, sources, free, free_count, P, table_out=None):
    """The outputs of one fork as a dict; inputs are not changed.  table_out: what the entries that are not written hold."""
    B, max_pages = table.shape
    pages = len(free)
    lengths = [max(int(x), 0) for x in lengths]
    out = (np.full_like(table, -1) if table_out is None else table_out).copy()
    free = free.copy()
    copies = np.full((B, 2), -1, np.int32)

    def nothing(status):
        for b in range(B):
            n = min(held(lengths[b], P), max_pages)
            out[b, :n] = table[b, :n]
        return dict(table=out, lengths=np.array(lengths, np.int32), free=free, free_left=int(free_count), copies=copies,
                    report=[status, 0, 0, max(lengths)])
    if max(int(s) for s in sources) >= B:
        return nothing(1)
    if max(lengths) > max_pages * P:
        return nothing(3)
    before = {int(p) for b in range(B) for p in table[b, :held(lengths[b], P)]}
    new_len = [lengths[s] if s >= 0 else 0 for s in sources]
    rows = [list(map(int, table[s, :held(lengths[s], P)])) if s >= 0 else [] for s in sources]
    # A page that a row fills in part is appended to: of the rows that go on with it one keeps it (one that stays itself, else
    # any; the lowest), and none where a row that goes on has it as a full page.
    full = {int(p) for s in sources if s >= 0 for p in table[s, :lengths[s] // P] if 0 <= p < pages}
    parts = {}
    for b in range(B):
        if new_len[b] % P:
            page = rows[b][-1]
            parts.setdefault((page,) if 0 <= page < pages else (page, int(sources[b])), []).append(b)
    need = []
    for key, held_by in parts.items():
        keeper = None if key[0] in full else min(held_by, key=lambda b: (sources[b] != b, b))
        need += [b for b in held_by if b != keeper]
    need.sort()
    after = {p for b in range(B) for p in (rows[b][:-1] if b in need else rows[b])}
    back = sorted(p for p in before - after if 0 <= p < pages)
    stack = [int(x) for x in free[:free_count]] + back
    if len(need) > len(stack) or len(stack) > pages:
        return nothing(3)
    free[:len(stack)] = stack
    for b in need:
        copies[b] = rows[b][-1], stack[-1]
        rows[b][-1] = stack.pop()
    for b in range(B):
        out[b, :len(rows[b])] = rows[b]
    return dict(table=out, lengths=np.array(new_len, np.int32), free=free, free_left=len(stack), copies=copies,
                report=[0, len(back), len(need), max(new_len)])


def compact(table, lengths, num_pages, P, max_moves, table_out=None, free=None):
    """The outputs of one compaction as a dict."""
    B, max_pages = table.shape
    lengths = [max(int(x), 0) for x in lengths]
    out = (np.full_like(table, -1) if table_out is None else table_out).copy()
    free = (np.full(num_pages, -1, np.int32) if free is None else free).copy()
    moves = np.full((max_moves, 2), -1, np.int32)
    if max(lengths) > max_pages * P:
        for b in range(B):
            n = min(held(lengths[b], P), max_pages)
            out[b, :n] = table[b, :n]
        return dict(table=out, free=free, free_left=None, moves=moves, report=[3, 0, 0, max(lengths)])
    live = sorted({int(p) for b in range(B) for p in table[b, :held(lengths[b], P)] if 0 <= p < num_pages})
    L = len(live)
    high = [p for p in live if p >= L]
    holes = sorted(set(range(L)) - set(live))
    goes = dict(zip(high, holes))
    moves[:len(high)] = np.array(list(goes.items()), np.int32).reshape(-1, 2)
    for b in range(B):
        n = held(lengths[b], P)
        out[b, :n] = [goes.get(int(p), int(p)) for p in table[b, :n]]
    free[:num_pages - L] = np.arange(num_pages - 1, L - 1, -1)
    return dict(table=out, free=free, free_left=num_pages - L, moves=moves, report=[0, len(high), L, max(lengths)])
