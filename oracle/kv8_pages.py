"""The book of the 8-bit cache's pages: refs int32 [pages] (table entries that hold each page), table int32
[rows][entries], -1 for none, GONE where a fork's prefix ends in a page that its parent had given back.  Every call updates both in place and returns the pairs of `moves`, the first
(count, short) among them.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np

GONE = -2


def _free(refs):
    return [p for p in range(len(refs)) if refs[p] <= 0]


def _is_page(p, refs):
    return 0 <= p < len(refs)


def _entries(tokens, page_size):
    return -(-max(int(tokens), 0) // page_size)


def grow(refs, table, page_size, lens):
    want = [_entries(n, page_size) for n in lens]
    if any(w > table.shape[1] for w in want):
        return [(0, -1)]
    places = []
    for b, w in enumerate(want):
        held = [e for e in range(w) if _is_page(table[b, e], refs) or table[b, e] == GONE]
        places += [(b, e) for e in range(held[-1] + 1 if held else 0, w)]
    free = _free(refs)
    if len(places) > len(free):
        return [(0, len(places) - len(free))]
    for place, p in zip(places, free):
        table[place] = p
        refs[p] = 1
    return [(len(places), 0)]


def fork(refs, table, page_size, parents, children, lens):
    rows, stride = table.shape
    none = [(-1, -1)] * len(parents)
    real = [i for i in range(len(parents)) if parents[i] >= 0 and children[i] >= 0]
    kids = [int(children[i]) for i in real]
    if any(parents[i] >= rows or children[i] >= rows or lens[i] < 0 or _entries(lens[i], page_size) > stride for i in real) \
            or len(set(kids)) < len(kids) or set(kids) & {int(parents[i]) for i in real}:
        return [(0, -1)] + none
    split = [i for i in real if lens[i] % page_size and _is_page(table[parents[i], lens[i] // page_size], refs)]
    free = _free(refs)
    if len(split) > len(free):
        return [(0, len(split) - len(free))] + none
    moves, before = list(none), table.copy()
    for i, p in zip(split, free):
        moves[i] = (int(before[parents[i], lens[i] // page_size]), p)
        refs[p] = 1
    for i in real:
        full = int(lens[i]) // page_size
        for p in before[children[i]]:
            if _is_page(p, refs):
                refs[p] -= 1
        row = np.full(stride, -1, np.int32)
        for e in range(full):
            p = before[parents[i], e]
            if _is_page(p, refs):
                row[e] = p
                refs[p] += 1
        if moves[i][1] >= 0:
            row[full] = moves[i][1]
        last = _entries(lens[i], page_size) - 1
        if last >= 0 and row[last] < 0:
            row[last] = GONE
        table[children[i]] = row
    return [(len(parents), 0)] + moves


def free(refs, table, page_size, rows, begin=None, end=None):
    for i, b in enumerate(rows):
        if not 0 <= b < len(table):
            continue
        for e in range(table.shape[1]):
            if (begin is None or e * page_size >= begin[i]) and (end is None or (e + 1) * page_size <= end[i]):
                if _is_page(table[b, e], refs):
                    refs[table[b, e]] -= 1
                table[b, e] = -1


def compact(refs, table, most):
    used = [p for p in reversed(range(len(refs))) if refs[p] > 0]
    moves = [(u, f) for u, f in zip(used, _free(refs)) if u > f][:most]
    to = dict(moves)
    for u, f in moves:
        refs[f], refs[u] = refs[u], 0
    for place, p in np.ndenumerate(table):
        table[place] = to.get(int(p), p)
    return [(len(moves), 0)] + moves + [(-1, -1)] * (most - len(moves))
