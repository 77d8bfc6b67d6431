"""Pages of the NVFP4 key/value cache between two tokens: fork, trim, compact.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

One sequence, one entry, one page at a time, with lists; the cache's buffers are numpy
uint8 arrays as in ``oracle.kv_cache``.
"""
from __future__ import annotations

import numpy as np


def _length(n, table, page):
    return min(max(int(n), 0), len(table) * page)


def _used(n, page):
    return -(-n // page)


def fork(cache, refs, tables, lens, parents, new_tokens, new_lens=None):
    """-> (tables, lens, refs, slots, cache, short): `short` where pages or table entries ran out."""
    page, pages = cache[0].shape[2], len(refs)
    refs, most = [int(r) for r in refs], tables.shape[1]
    held = lambda p: 0 <= p < pages                                          # noqa: E731
    olds = [(list(map(int, t)), _length(n, t, page)) for t, n in zip(tables, lens)]
    for t, n in olds:
        for p in t[: _used(n, page)]:
            if held(p):
                refs[p] -= 1
    short, kids, writers = False, [], {}
    for i, par in enumerate(parents):
        if not 0 <= par < len(olds):
            kids.append(([], 0, 0))
            continue
        t, n = olds[par]
        more = new_tokens if new_lens is None else min(max(int(new_lens[i]), 0), new_tokens)
        m = min(n + more, most * page)
        short |= m < n + more
        mine = t[: _used(n, page)]
        kids.append((mine, n, m))
        for idx, p in enumerate(mine):
            if not held(p):
                continue
            if (idx + 1) * page > n and m > n:                               # about to be written
                writers.setdefault(p, []).append(i)
            else:
                refs[p] += 1
    stays = {}                                                              # page -> the child that keeps it
    for p, who in writers.items():
        if refs[p] <= 0:
            stays[p] = min(who)
            refs[p] = 1
    free = [p for p in range(pages) if refs[p] <= 0]
    refs = [max(r, 0) for r in refs]
    new = [c.copy() for c in cache]

    def take():
        nonlocal short
        if not free:
            short = True
            return -1
        refs[free[0]] = 1
        return free.pop(0)
    out = np.full((len(kids), most), -1, np.int64)
    slots = np.full((len(kids), new_tokens), -1, np.int64)
    for i, (mine, n, m) in enumerate(kids):
        mine = list(mine)
        if n % page and m > n and held(mine[-1]) and stays.get(mine[-1]) != i:
            src, mine[-1] = mine[-1], take()
            g = -(-(n % page) // 16) * 16
            if mine[-1] >= 0:
                for k in range(3):
                    new[k][mine[-1], :, :g] = cache[k][src, :, :g]
                new[3][mine[-1], :, :, :g] = cache[3][src, :, :, :g]
        while len(mine) < _used(m, page):
            mine.append(take())
        out[i, : len(mine)] = mine
        for x in range(n, min(m, n + new_tokens)):
            if held(mine[x // page]):
                slots[i, x - n] = mine[x // page] * page + x % page
    return out, np.array([m for _, _, m in kids], np.int64), np.array(refs, np.int64), slots, new, short


def trim(page, refs, tables, lens, first=None, end=None):
    refs, pages, most = [int(r) for r in refs], len(refs), tables.shape[1]
    out, ends = np.full(tables.shape, -1, np.int64), []
    for b, t in enumerate(tables):
        n = _length(lens[b], t, page)
        lo = 0 if first is None else max(int(first[b]), 0)
        hi = n if end is None else min(max(int(end[b]), 0), n)
        ends.append(hi)
        for i in range(min(_used(n, page), most)):
            p = int(t[i])
            if not 0 <= p < pages:
                continue
            if lo // page <= i < _used(hi, page):
                out[b, i] = p
            else:
                refs[p] -= 1
    return out, np.array(ends, np.int64), np.array(refs, np.int64)


def compact(cache, refs, tables, lens):
    """-> (tables, refs, map, live, cache)."""
    page, pages = cache[0].shape[2], len(refs)
    live = [p for p in range(pages) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    to = {p: p if p < n else holes.pop(0) for p in live}
    new = [c.copy() for c in cache]
    out_refs = np.zeros(pages, np.int64)
    for p, q in to.items():
        out_refs[q] = refs[p]
        for k in range(4):
            new[k][q] = cache[k][p]
    out = np.full(tables.shape, -1, np.int64)
    for b, t in enumerate(tables):
        for i in range(_used(_length(lens[b], t, page), page)):
            out[b, i] = to.get(int(t[i]), -1)
    return out, out_refs, np.array([to.get(p, -1) for p in range(pages)], np.int64), n, new
