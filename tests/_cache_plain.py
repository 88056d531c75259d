"""The paged cache's upkeep on Python lists: what attn_cache_* have to do, one
sequence after the other.  State: table rows (lists), lens, refs (lists); pools as
numpy arrays [layers][num_pages][page][row]."""


def pages(n, page):
    return -(-n // page)


def reorder(table, lens, refs, index, page):
    refs = list(refs)
    rows = [table[i][:pages(lens[i], page)] if i >= 0 else [] for i in index]
    for row in rows:
        for p in row:
            refs[p] += 1
    for row, n in zip(table, lens):
        for p in row[:pages(n, page)]:
            refs[p] -= 1
    return rows, [lens[i] if i >= 0 else 0 for i in index], refs


def reserve(pools, table, lens, refs, add, page, width):
    """-> (rows, lens, refs, free); pools are changed in place."""
    rows = [row[:pages(n, page)] for row, n in zip(table, lens)]
    if any(pages(n + a, page) > width for n, a in zip(lens, add)):
        return rows, list(lens), list(refs), -len(refs) - 1
    free = [p for p, r in enumerate(refs) if r == 0]
    left, out, copies, need = list(refs), list(refs), [], 0
    new = [list(r) for r in rows]
    for b, (n, a) in enumerate(zip(lens, add)):
        old = None
        if a > 0 and n % page and left[new[b][-1]] > 1:
            old = new[b].pop()
            left[old] -= 1
        while len(new[b]) < pages(n + a, page):
            new[b].append(free[need] if need < len(free) else -1)
            if old is not None:
                copies.append((old, new[b][-1]))
                old = None
            need += 1
    if need > len(free):
        return rows, list(lens), list(refs), len(free) - need
    for src, dst in copies:
        out[src] -= 1
        for pool in pools:
            pool[:, dst] = pool[:, src]
    for p in free[:need]:
        out[p] = 1
    return new, [n + a for n, a in zip(lens, add)], out, len(free) - need


def accept(pools, table, lens, refs, path, tree, page):
    """path: a list of accepted nodes per sequence."""
    refs, out = list(refs), []
    for row, n, keep, t in zip(table, lens, path, tree):
        t = min(t, n)
        base = n - t
        for pool in pools:
            old = [pool[:, row[(base + x) // page], (base + x) % page].copy() for x in keep]
            for i, x in enumerate(old):
                pool[:, row[(base + i) // page], (base + i) % page] = x
        out.append(base + len(keep))
        for p in row[pages(out[-1], page):pages(n, page)]:
            refs[p] -= 1
    return out, refs


def compact(pools, table, lens, refs, page):
    n = sum(r > 0 for r in refs)
    holes = iter([p for p in range(n) if refs[p] <= 0])
    go = [-1 if r <= 0 else p if p < n else next(holes) for p, r in enumerate(refs)]
    after = [0] * len(refs)
    for p, to in enumerate(go):
        if to >= 0:
            after[to] = refs[p]
            if to != p:
                for pool in pools:
                    pool[:, to] = pool[:, p]
    return [[go[p] for p in row[:pages(k, page)]] for row, k in zip(table, lens)], after, go
