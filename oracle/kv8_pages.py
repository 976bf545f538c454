"""The pages of a paged cache: reserve, fork, free, compact and copy on lists.

A pool is dict(refs [P], table [B][width], lens [B], T); a page's contents are
whatever `moves` (pairs (from, to), carried out in order) brings there.  The
functions change the pool in place and return (status, moves).
"""


def held(pool, b):
    """The table entries of row b that count."""
    T, width = pool["T"], len(pool["table"][b])
    return pool["table"][b][:min(-(-max(pool["lens"][b], 0) // T), width)]


def length(pool, b):
    return min(max(pool["lens"][b], 0), len(pool["table"][b]) * pool["T"])


def free(pool, rows):
    for b in rows:
        if not 0 <= b < len(pool["lens"]):
            continue
        pages = held(pool, b)
        for i, p in enumerate(pages):
            if 0 <= p < len(pool["refs"]):
                pool["refs"][p] -= 1
            pool["table"][b][i] = -1
        pool["lens"][b] = 0
    return 0, []


def reserve(pool, added):
    T, free_pages = pool["T"], [p for p, n in enumerate(pool["refs"]) if n == 0]
    wants = []
    for b, n in enumerate(added):
        old = length(pool, b)
        new = max(old + n, 0)
        if new > len(pool["table"][b]) * T:
            return -1, []
        if n < 0 and new % T:
            p = pool["table"][b][new // T]
            if 0 <= p < len(pool["refs"]) and pool["refs"][p] > 1:
                return -1, []
        wants += [(b, i) for i in range(-(-old // T), -(-new // T))]
    if len(wants) > len(free_pages):
        return len(wants) - len(free_pages), []
    for (b, i), p in zip(wants, free_pages):
        pool["table"][b][i] = p
        pool["refs"][p] = 1
    for b, n in enumerate(added):
        old = length(pool, b)
        pool["lens"][b] = max(old + n, 0)
        for i in range(-(-pool["lens"][b] // T), -(-old // T)):
            if 0 <= pool["table"][b][i] < len(pool["refs"]):
                pool["refs"][pool["table"][b][i]] -= 1
            pool["table"][b][i] = -1
    return 0, []


def fork(pool, src, dst):
    B, T = len(pool["lens"]), pool["T"]
    bad = any(not 0 <= r < B for r in [*src, *dst]) or len(set(dst)) < len(dst) or set(src) & set(dst)
    if bad or any(length(pool, d) for d in dst):
        return -1, []
    free_pages = [p for p, n in enumerate(pool["refs"]) if n == 0]
    short = sum(length(pool, s) % T != 0 for s in src) - len(free_pages)
    if short > 0:
        return short, []
    moves = []
    for s, d in zip(src, dst):
        L = length(pool, s)
        for i in range(L // T):
            p = pool["table"][d][i] = pool["table"][s][i]
            if 0 <= p < len(pool["refs"]):
                pool["refs"][p] += 1
        if L % T:
            p = pool["table"][d][L // T] = free_pages.pop(0)
            pool["refs"][p] = 1
            moves.append((pool["table"][s][L // T], p))
        pool["lens"][d] = L
    return 0, moves


def compact(pool):
    refs = pool["refs"]
    used = sum(n > 0 for n in refs)
    moves = list(zip((p for p in range(used, len(refs)) if refs[p] > 0),
                     (p for p in range(used) if refs[p] <= 0)))
    to = dict(moves)
    for b in range(len(pool["lens"])):
        for i, p in enumerate(held(pool, b)):
            pool["table"][b][i] = to.get(p, p)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    return used, moves
