"""Oracle: accepted drafts moved together, and the page pool, in plain Python, entry by entry.

Test infrastructure only (see the package docstring).  The definitions are this library's [DEF]: a row of a page table holds
its leading entries in [0, num_pages), refs counts the rows that hold a page, free pages are handed out lowest first.
"""

import numpy as np


def accepted_ref(path_row):
    """How many entries of a path are accepted: up to the first that is negative or does not increase."""
    n, before = 0, -1
    for e in path_row:
        if e <= before:
            break
        n, before = n + 1, int(e)
    return n


def compact_ref(planes, table, start, path, page_size, num_pages):
    """planes: arrays [slots, ...], changed in place.  Returns the new lengths."""
    lengths = []
    for b in range(len(start)):
        def slot(pos):
            p = pos // page_size
            page = int(table[b][p]) if pos >= 0 and p < len(table[b]) else -1
            return page * page_size + pos % page_size if 0 <= page < num_pages else -1
        n = accepted_ref(path[b])
        moves = [(slot(int(start[b]) + int(path[b][i])), slot(int(start[b]) + i)) for i in range(n)]
        moves = [(s, d) for s, d in moves if s >= 0 and d >= 0]
        for a in planes:
            held = [a[s].copy() for s, _ in moves]
            for (_, d), x in zip(moves, held):
                a[d] = x
        lengths.append(int(start[b]) + n)
    return lengths


def held_ref(row, num_pages):
    n = 0
    while n < len(row) and 0 <= row[n] < num_pages:
        n += 1
    return n


def _take(refs, wants):
    """wants: (row of the table, column) in order.  Returns the page for each, -1 where none is free any more."""
    free = [int(p) for p in np.flatnonzero(refs <= 0)]
    return [free[i] if i < len(free) else -1 for i in range(len(wants))]


def _copy(planes, page_size, copies):
    for src, dst, rows in copies:
        for a in planes:
            a[dst * page_size:dst * page_size + rows] = a[src * page_size:src * page_size + rows]


def resize_ref(refs, table, lengths, page_size, planes=()):
    """refs [num_pages], table [rows, columns] and planes change in place.  Returns the pages that were missing."""
    N, width = len(refs), table.shape[1]
    for b, n in enumerate(lengths):
        if n < 0:
            continue
        want = min(-(-int(n) // page_size), width)
        held = held_ref(table[b], N)
        for i in range(want, width):
            if i < held:
                refs[table[b, i]] -= 1
            table[b, i] = -1
    wants = []
    for b, n in enumerate(lengths):
        if n < 0:
            continue
        want = min(-(-int(n) // page_size), width)
        held = held_ref(table[b], N)
        if held < want:
            wants += [(b, i, None) for i in range(held, want)]
        elif want and n % page_size and n < width * page_size and refs[table[b, want - 1]] > 1:
            wants.append((b, want - 1, int(table[b, want - 1])))
    pages = _take(refs, wants)
    copies, missing = [], 0
    for (b, i, old), page in zip(wants, pages):
        if page < 0:
            if old is not None:
                if refs[old] == 1:  # the others have let go of it: it is the row's own
                    continue
                refs[old] -= 1
            missing += 1
            table[b, i] = -1
            continue
        table[b, i] = page
        refs[page] = 1
        if old is not None:
            refs[old] -= 1
            copies.append((old, page, int(lengths[b]) % page_size))
    _copy(planes, page_size, copies)
    return missing


def fork_ref(refs, table, src, dst, lengths, page_size, planes=()):
    """As resize_ref."""
    N, (rows, width) = len(refs), table.shape
    sources, seen, wants = {int(s) for s in src}, set(), []
    before = table.copy()  # sources are no pair's destination: their rows do not change
    for s, d, n in zip(map(int, src), map(int, dst), map(int, lengths)):
        again = d in seen
        seen.add(d)
        if again or d in sources or not (0 <= s < rows and 0 <= d < rows) or n < 0:
            continue
        for i in range(held_ref(before[d], N)):
            refs[before[d, i]] -= 1
        table[d] = -1
        held, whole = held_ref(before[s], N), n // page_size
        for i in range(min(whole, held)):
            table[d, i] = before[s, i]
            refs[before[s, i]] += 1
        if n % page_size and whole < held:
            wants.append((d, whole, int(before[s, whole]), n % page_size))
    pages = _take(refs, wants)
    copies, missing = [], 0
    for (d, i, old, n), page in zip(wants, pages):
        if page < 0:
            missing += 1
            continue
        table[d, i] = page
        refs[page] = 1
        copies.append((old, page, n))
    _copy(planes, page_size, copies)
    return missing
