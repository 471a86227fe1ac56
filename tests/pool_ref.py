"""Plain restatement (numpy, page by page) of the calls on the pool of cache pages, for the tests.
Written from the definitions in include/osm_attn.h.  Every function changes its arrays in place and
returns whether something is to be reported."""
import numpy as np


def count(tokens, P):
    return (tokens + P - 1) // P


def clamp(n, table, P):
    return min(max(int(n), 0), table.shape[1] * P)


class Free:
    """Hands out the lowest free pages of what refs were at first."""

    def __init__(self, refs):
        self.ids = [p for p in range(len(refs)) if refs[p] <= 0]
        self.ran_out = False

    def next(self):
        if not self.ids:
            self.ran_out = True
            return -1
        return self.ids.pop(0)


def grow(table, lens, new_lens, refs, P):
    """Returns (old_lens, copies, bad): copies the (from page, to page, tokens)."""
    free, old, copies, uses = Free(refs), [], [], refs.copy()
    for b in range(len(lens)):
        had = clamp(lens[b], table, P)
        has = clamp(had + max(int(new_lens[b]), 0), table, P)
        old.append(had)
        lens[b] = has
        if has > had and had % P:
            e = table[b, had // P]
            if 0 <= e < len(refs) and uses[e] > 1:
                p = free.next()
                table[b, had // P] = p
                refs[e] -= 1
                if p >= 0:
                    refs[p] = 1
                    copies.append((int(e), p, had % P))
        for j in range(count(had, P), count(has, P)):
            p = free.next()
            table[b, j] = p
            if p >= 0:
                refs[p] = 1
    return np.array(old, dtype=np.int32), copies, free.ran_out


def fork(table, lens, refs, P, src, dst):
    before, bad, rows, taken = lens.copy(), False, table.copy(), set()
    for s, t in zip(map(int, src), map(int, dst)):
        if s < 0 or t < 0:
            continue
        if s >= len(lens) or t >= len(lens) or before[t] > 0 or t in taken:
            bad = True
            continue
        taken.add(t)
        lens[t] = clamp(before[s], table, P)
        for j in range(count(lens[t], P)):
            table[t, j] = rows[s, j]
            if 0 <= rows[s, j] < len(refs):
                refs[rows[s, j]] += 1
    return bad


def release(table, lens, refs, P, rows, keep):
    bad = False
    for r, k in zip(map(int, rows), map(int, keep)):
        if r < 0:
            continue
        if r >= len(lens):
            bad = True
            continue
        k = max(k, 0)
        for j in range(count(k, P), count(clamp(lens[r], table, P), P)):
            p = table[r, j]
            if 0 <= p < len(refs):
                refs[p] = max(refs[p] - 1, 0)
        lens[r] = min(int(lens[r]), k)
    return bad


def compact(table, lens, refs, P):
    """Returns (page_map, used, moves)."""
    used = int((refs > 0).sum())
    holes = [p for p in range(used) if refs[p] <= 0]
    movers = [p for p in range(used, len(refs)) if refs[p] > 0]
    where = np.array([p if r > 0 else -1 for p, r in enumerate(refs)], dtype=np.int32)
    for a, b in zip(movers, holes):
        where[a] = b
        refs[b], refs[a] = refs[a], 0
    for b in range(len(lens)):
        for j in range(count(clamp(lens[b], table, P), P)):
            if 0 <= table[b, j] < len(refs):
                table[b, j] = where[table[b, j]]
    return where, used, list(zip(movers, holes))
