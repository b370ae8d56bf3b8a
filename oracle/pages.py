"""Oracle of the page pool: the calls' definitions as sequential host loops
over a reference count per page.  Each returns the set of error codes a call
may report first.

TEST INFRASTRUCTURE ONLY, as the rest of this package.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
DEVICE_INPUT, NO_PAGES = 5, 7


def _free(ref):
    return [int(p) for p in np.flatnonzero(np.asarray(ref) == 0)]


def alloc(ref, table, begin, end, full_only):
    """Rows in order; a row that does not fit after the demands before it gets
    nothing."""
    errors, free, asked = set(), _free(ref), 0
    width = table.shape[1]
    for b in range(len(table)):
        f, t = (0 if begin is None else int(begin[b])), int(end[b])
        if not 0 <= f <= t <= width * PAGE:
            errors.add(DEVICE_INPUT)
            continue
        want = [i for i in range(f // PAGE, t // PAGE if full_only else -(-t // PAGE)) if table[b, i] == -1]
        if want and asked + len(want) > len(free):
            errors.add(NO_PAGES)
        else:
            for k, i in enumerate(want):
                table[b, i] = free[asked + k]
                ref[free[asked + k]] = 1
        asked += len(want)
    return errors


def fork(ref, table, src, dst, length, full_only):
    errors, free, asked = set(), _free(ref), 0
    B, width = table.shape
    old_ref, old = ref.copy(), table.copy()
    copies = [(-1, -1)] * len(src)

    def sound(i):
        return 0 <= src[i] < B and 0 <= dst[i] < B and src[i] != dst[i] and 0 <= length[i] <= width * PAGE

    into = {}
    for i in range(len(src)):
        if sound(i):
            into.setdefault(int(dst[i]), i)
    for i in range(len(src)):
        ok = sound(i) and into[int(dst[i])] == i and int(src[i]) not in into
        if ok:
            full = int(length[i]) // PAGE
            part = not full_only and length[i] % PAGE != 0
            ok = (old[dst[i]] == -1).all()
            for e in range(full + part):
                p = old[src[i], e]
                if p == -1:
                    ok = ok and e != full
                else:
                    ok = ok and 0 <= p < len(ref) and old_ref[p] > 0
        if not ok:
            errors.add(DEVICE_INPUT)
            continue
        if part:
            asked += 1
            if asked > len(free):
                errors.add(NO_PAGES)
                continue
        for e in range(full):
            if old[src[i], e] >= 0:
                ref[old[src[i], e]] += 1
                table[dst[i], e] = old[src[i], e]
        if part:
            p = free[asked - 1]
            ref[p] = 1
            table[dst[i], full] = p
            copies[i] = (int(old[src[i], full]), p)
    return errors, np.asarray(copies, dtype=np.int32).reshape(-1, 2)


def trim(ref, table, keep_begin, keep_end):
    errors = set()
    B, width = table.shape
    for b in range(B):
        f, t = (0 if keep_begin is None else int(keep_begin[b])), int(keep_end[b])
        if not 0 <= f <= t <= width * PAGE:
            errors.add(DEVICE_INPUT)
            continue
        for e in range(width):
            p = int(table[b, e])
            if f // PAGE <= e < -(-t // PAGE) or p == -1:
                continue
            table[b, e] = -1
            if not 0 <= p < len(ref) or ref[p] <= 0:
                errors.add(DEVICE_INPUT)
            else:
                ref[p] -= 1
    return errors


def compact(ref, table):
    """(errors, new table, new reference counts, [(src, dst)])."""
    errors = set()
    used = [p for p in range(len(ref)) if ref[p] > 0]
    U = len(used)
    movers = [p for p in used if p >= U]
    holes = [p for p in range(U) if ref[p] <= 0]
    to = {p: p for p in used if p < U}
    to.update(zip(movers, holes))
    new_ref, new_table = np.zeros_like(ref), np.full_like(table, -1)
    for p in used:
        new_ref[to[p]] = ref[p]
    for i, p in np.ndenumerate(table):
        if p == -1:
            continue
        if int(p) in to:
            new_table[i] = to[int(p)]
        else:
            errors.add(DEVICE_INPUT)
    return errors, new_table, new_ref, list(zip(movers, holes))
