"""The page table's operators on the host, page by page, as the oracle of
mla_pages_fork and mla_pages_compact."""
import numpy as np

PAGE = 64


def pages_of(n):
    return -(-n // PAGE)


def table_of(rows, stride):
    """Page lists -> int32 [R, stride] of slots; -7 where a row has no page."""
    t = np.full((len(rows), stride), -7, np.int32)
    for i, row in enumerate(rows):
        e = (np.asarray(row, np.int64)[:, None] * PAGE + np.arange(PAGE)).reshape(-1)[:stride]
        t[i, :len(e)] = e
    return t


def counts(rows, num_pages):
    refs = np.zeros(num_pages, np.int32)
    for row in rows:
        for p in row:
            refs[p] += 1
    return refs


def fork(rows, lens, refs, parents, keep, grow):
    """rows: page lists.  Returns (new rows, new lens, refs, copies [3, R]) or None
    when there are too few pages."""
    R, refs = len(rows), refs.copy()
    taken = [0 if parents[i] < 0 else min(keep[i], lens[parents[i]]) for i in range(R)]
    new, copies = [], np.array([[-1] * R, [-1] * R, [0] * R], np.int32)
    free = [p for p in range(1, len(refs)) if refs[p] == 0]
    after = np.zeros_like(refs)
    at = 0
    need = 0
    for i in range(R):
        full, part = divmod(taken[i], PAGE)
        p = parents[i]
        row = list(rows[p][:full]) if p >= 0 else []
        if part:
            page = rows[p][full]
            # who else wants this page: another row, or another child of the same parent
            others = [j for j in range(R) if j != i and parents[j] == p and
                      (taken[j] // PAGE > full or (taken[j] // PAGE == full and taken[j] % PAGE and j < i))]
            if refs[page] == 1 and not others:
                row.append(page)
            else:
                if at < len(free):
                    copies[:, i] = page, free[at], part
                    row.append(free[at])
                at += 1
        while len(row) < pages_of(taken[i] + grow[i]) and at < len(free) + 1:
            if at < len(free):
                row.append(free[at])
            else:
                need = 1
                break
            at += 1
        new.append(row)
    if at > len(free) or need:
        return None
    for row in new:
        for p in row:
            after[p] += 1
    # rows outside this table hold the rest
    outside = refs - counts(rows, len(refs))
    return new, [taken[i] + grow[i] for i in range(R)], after + outside, copies


def compact(rows, refs, max_moves):
    """Returns (new rows, refs, src, dst)."""
    refs = refs.copy()
    live = [p for p in range(1, len(refs)) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(1, n + 1) if refs[p] == 0]
    high = [p for p in reversed(live) if p > n]
    assert len(holes) == len(high)
    m = min(len(holes), max_moves)
    to = dict(zip(high[:m], holes[:m]))
    for s, d in to.items():
        refs[d], refs[s] = refs[s], 0
    return [[to.get(p, p) for p in row] for row in rows], refs, high[:m], holes[:m]
